// Residual layer norm with an optional 8-bit output, and whole rows to 8-bit
// integers, which is the same kernel without the norm.
//
//   h = x + residual      mean = sum_j h / d     v = h - mean
//   rstd = 1 / sqrt(mean_j v^2 + eps)            n = v rstd w + b
//   y = n, rounded once, or q = n / scale in e4m3 or int8, rounded once, with
//   scale = max_j |n| / 448 or / 127
//
// The statistics are of the fp32 sum x + residual. The variance is a sum of
// squares about means, which keeps its digits where the mean is far larger than
// the spread (a sum of h^2 would lose them all).
//
// HBM bound, as the RMS norm, whose row loads, shapes and grids these kernels
// share: a row is read once into the registers of one wave or one workgroup.
// Measured: 8192 x 8192 bf16 with a residual to h and int8 rows 83 us, 5.7 TB/s
// (the RMS norm to e4m3 79); one row of 8192 4.0 us on the GPU; whole rows of
// 8192 x 8192 to int8 38 us. Rows of 1024 threads took 104 to 118 us where 512
// took 84 to 92.
#pragma once

#include "dora_launch.h"
#include "dora_rows.h"

namespace dora {

namespace {

struct LayerNormArgs {
  const void* x;
  const void* residual;
  const float* weight;
  const float* bias;
  float eps;
  int64_t T, d;
  void* h;
  void* y;
  void* q;
  int q8;        // q holds e4m3 (kQE4m3) or integers (kQInt8)
  float* scale;
  float* mean;
  float* rstd;
};

// E biases of a chunk; zeros where there are none and past d.
template <int E>
__device__ __forceinline__ void load_bias(const float* b, int64_t k, int64_t d, float (&f)[E]) {
  if (b == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 0.f;
  } else {
    load_weight<E>(b, k, d, f);
  }
}

// How many of a chunk's elements [k, k + E) lie in a row of d.
template <int E>
__device__ __forceinline__ int chunk_left(int64_t k, int64_t d) {
  const int64_t left = d - k;
  return (int)(left < E ? left : E);
}

// The same address, which the compiler takes for another: what is read there in
// a loop stays in it.
__device__ __forceinline__ const float* reread(const float* p) {
  asm volatile("" : "+s"(p));
  return p;
}

// The spread of a row whose squares about its mean add up to q. A NaN or an infinity
// in the row, or a sum past fp32's range, leaves a q that is no finite number, and
// both statistics are then NaN (1 / sqrt(inf) would be 0, and such a row its bias).
__device__ __forceinline__ void finish_stats(float q, int64_t d, float eps, float& mean, float& rstd) {
  const bool fine = q <= 3.402823466e38f;
  rstd = fine ? 1.f / sqrtf(q / (float)d + eps) : __builtin_nanf("");
  mean = fine ? mean : __builtin_nanf("");
}

// The row's statistics, from the C chunks that each of NT threads holds; past d
// the values do not count. Each wave takes the mean of its own values and their
// squares about it; the waves' (count, mean, squares) join as those of any
// parts do: the squares about the whole mean are the parts' own and count times
// the square of each part's distance to it (Chan, Golub, LeVeque 1979). One
// exchange between the waves serves both; a part's mean is off by a few 2^-24 of
// itself, which counts times its distance to the whole one.
template <int NT, int C, int E>
__device__ __forceinline__ void row_stats(const float (&f)[C][E], int lane, int64_t d, float eps, float* red,
                                          float& mean, float& rstd) {
  constexpr int W = NT / 64;
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) s += f[c][e];
  // values of wave w
  auto count = [&](int w) __attribute__((always_inline)) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t left = d - (int64_t)(c * NT + w * 64) * E;
      n += left < 0 ? 0 : (left < 64 * E ? (int)left : 64 * E);
    }
    return (float)n;
  };
  const int wave = W > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const float own = count(wave);
  const float mu = own > 0.f ? wave_sum(s) / own : 0.f;
  float q = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int n = chunk_left<E>((int64_t)(c * NT + lane) * E, d);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = e < n ? f[c][e] - mu : 0.f;
      q = fmaf(v, v, q);
    }
  }
  q = wave_sum(q);
  mean = mu;
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) red[2 * wave] = mu, red[2 * wave + 1] = q;
    __syncthreads();
    // (lane w % 16 takes wave w's, so that each row of 16 lanes holds them all)
    static_assert(W <= 16, "the waves of a workgroup are lanes of a row of 16");
    const int w = threadIdx.x & 15;
    const float n = w < W ? count(w) : 0.f, m = w < W ? red[2 * w] : 0.f;
    mean = row16_sum(n * m) / (float)d;
    q = row16_sum(fmaf(n * (m - mean), m - mean, w < W ? red[2 * w + 1] : 0.f));
  }
  finish_stats(q, d, eps, mean, rstd);
}

// Largest |value| of the row, as its bits (see row_max_bits).
template <int NT>
__device__ __forceinline__ uint32_t row_top(uint32_t v, uint32_t* lds) {
  v = wave_max(v);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    const int w = threadIdx.x & 15;
    v = row16_max(w < NT / 64 ? lds[w] : 0u);
  }
  return v;
}

// NT threads and C chunks a thread to a row; workgroups of 256 threads hold
// 256 / NT rows where NT is 64. A workgroup walks rows gridDim.x apart: its
// weights are read once, and a row's loads go out before the row ahead of it
// is reduced. NORM false: n is x itself.
template <typename T, int NT, int C, bool STREAM, bool LINES, bool NORM>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void layer_norm_kernel(LayerNormArgs a) {
  constexpr int E = Elem<T>::epc, W = NT > 64 ? NT / 64 : 1;
  // (two sets of words: a wave one row ahead uses the other one)
  __shared__ float red[2][3 * W];
  const int lane = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  constexpr int RPW = NT == 64 ? 4 : 1;   // rows a workgroup holds at a time
  int par = 0;
  const int64_t t0 = (int64_t)blockIdx.x * RPW + (NT == 64 ? threadIdx.x >> 6 : 0);
  const bool has_res = NORM && a.residual != nullptr;
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
  // (Four chunks of 1024 threads, which have 128 registers each: no row ahead, and
  // the weights are read anew for each row.)
  constexpr bool AHEAD = NT * C < 4096, KEEP = NORM && AHEAD;
  if (AHEAD && t0 < a.T) load(t0);
  float w[C][E], b[C][E];
  if constexpr (KEEP) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      load_weight<E>(a.weight, (int64_t)(c * NT + lane) * E, a.d, w[c]);
      load_bias<E>(a.bias, (int64_t)(c * NT + lane) * E, a.d, b[c]);
    }
  }
  for (int64_t t = t0; t < a.T; t += (int64_t)gridDim.x * RPW, par ^= 1) {
    if (!AHEAD) load(t);
    float f[C][E];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      unpack<T, E>(xv[c], f[c]);
      if (has_res) {
        float r[E];
        unpack<T, E>(rv[c], r);
#pragma unroll
        for (int e = 0; e < E; ++e) f[c][e] += r[e];
      }
    }
    // (h may be x or residual itself: other rows' loads are of other rows)
    if (AHEAD && t + (int64_t)gridDim.x * RPW < a.T) load(t + (int64_t)gridDim.x * RPW);
    if constexpr (NORM) {
      if (a.h) {
        T* h = static_cast<T*>(a.h) + t * a.d;
#pragma unroll
        for (int c = 0; c < C; ++c) store_row_chunk<T, STREAM>(h, (int64_t)(c * NT + lane) * E, a.d, f[c]);
      }
      float mean, rs;
      row_stats<NT, C, E>(f, lane, a.d, a.eps, red[par], mean, rs);
      if (lane == 0 && a.mean) a.mean[t] = mean;
      if (lane == 0 && a.rstd) a.rstd[t] = rs;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (!KEEP) {
          load_weight<E>(reread(a.weight), (int64_t)(c * NT + lane) * E, a.d, w[c]);
          load_bias<E>(reread(a.bias), (int64_t)(c * NT + lane) * E, a.d, b[c]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) f[c][e] = fmaf((f[c][e] - mean) * rs, w[c][e], b[c][e]);
      }
      if (a.y) {
        T* y = static_cast<T*>(a.y) + t * a.d;
#pragma unroll
        for (int c = 0; c < C; ++c) store_row_chunk<T, STREAM>(y, (int64_t)(c * NT + lane) * E, a.d, f[c]);
      }
    }
    if (a.q) {   // uniform over the grid
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int n = chunk_left<E>((int64_t)(c * NT + lane) * E, a.d);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t v = e < n ? abs_bits(f[c][e]) : 0u;
          top = v > top ? v : top;
        }
      }
      top = row_top<NT>(top, reinterpret_cast<uint32_t*>(red[par]) + 2 * (W - (NT == 64)));
      const float s = store_row_8<E, NT, C, STREAM>(static_cast<uint8_t*>(a.q) + t * a.d, lane, a.d, f, top, a.q8);
      if (lane == 0) a.scale[t] = s;
    }
  }
}

// Rows of any length: the row is read once for its mean, once for its
// variance, once for its largest |n| and once to be written (h is written
// last, so that it may be x or residual itself).
template <typename T, bool NORM>
__global__ __launch_bounds__(1024) void layer_norm_long_kernel(LayerNormArgs a) {
  constexpr int E = Elem<T>::epc, NT = 1024, W = NT / 64;
  __shared__ float red[2][3 * W];
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const T* x = static_cast<const T*>(a.x) + t * a.d;
    const T* res = NORM && a.residual ? static_cast<const T*>(a.residual) + t * a.d : nullptr;
    auto load = [&](int64_t k, float (&f)[E]) __attribute__((always_inline)) {
      unpack<T, E>(load_row_chunk(x, k, a.d), f);
      if (res) {
        float r[E];
        unpack<T, E>(load_row_chunk(res, k, a.d), r);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] += r[e];
      }
    };
    float mean = 0.f, rs = 1.f;
    if constexpr (NORM) {
      float s = 0.f, q = 0.f;
      for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
        float f[E];
        load(k, f);
#pragma unroll
        for (int e = 0; e < E; ++e) s += f[e];
      }
      mean = row_sum<NT>(s, red[par]) / (float)a.d;
      for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
        float f[E];
        load(k, f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float v = k + e < a.d ? f[e] - mean : 0.f;
          q = fmaf(v, v, q);
        }
      }
      finish_stats(row_sum<NT>(q, red[par] + W), a.d, a.eps, mean, rs);
      if (threadIdx.x == 0 && a.mean) a.mean[t] = mean;
      if (threadIdx.x == 0 && a.rstd) a.rstd[t] = rs;
    }
    auto normed = [&](int64_t k, float (&f)[E]) __attribute__((always_inline)) {
      if constexpr (NORM) {
        float w[E], b[E];
        load_weight<E>(a.weight, k, a.d, w);
        load_bias<E>(a.bias, k, a.d, b);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = fmaf((f[e] - mean) * rs, w[e], b[e]);
      }
    };
    uint32_t top = 0;
    if (a.q) {
      for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
        float f[E];
        load(k, f);
        normed(k, f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t v = k + e < a.d ? abs_bits(f[e]) : 0u;
          top = v > top ? v : top;
        }
      }
      top = row_max_bits<NT>(top, reinterpret_cast<uint32_t*>(red[par]) + 2 * W);
      if (threadIdx.x == 0) a.scale[t] = a.q8 == kQInt8 ? int8_scale_of(top) : scale_of(top);
    }
    for (int64_t k = (int64_t)threadIdx.x * E; k < a.d; k += NT * E) {
      float f[E];
      load(k, f);
      if (NORM && a.h) store_row_chunk<T>(static_cast<T*>(a.h) + t * a.d, k, a.d, f);
      normed(k, f);
      if (NORM && a.y) store_row_chunk<T>(static_cast<T*>(a.y) + t * a.d, k, a.d, f);
      // (one chunk of "lane" k / E)
      if (a.q) {
        const float(&one)[1][E] = reinterpret_cast<const float(&)[1][E]>(f);
        store_row_8<E, NT, 1, false>(static_cast<uint8_t*>(a.q) + t * a.d, (int)(k / E), a.d, one, top, a.q8);
      }
    }
  }
}

template <typename T, bool NORM>
hipError_t launch_fwd(const LayerNormArgs& a, hipStream_t st) {
  const RowShape r = forward_shape(a.T, a.d, Elem<T>::epc);
#define DORA_NORM(NT, C)                                                                                   \
  if (r.nt == NT && r.c == C) {                                                                            \
    const dim3 grid(grid_of(NT == 64 ? (a.T + 3) / 4 : a.T, NT)), block(NT == 64 ? 256 : NT);              \
    if (a.T * a.d * (int64_t)sizeof(T) <= kStreamBytes)                                                    \
      hipLaunchKernelGGL((layer_norm_kernel<T, NT, C, false, false, NORM>), grid, block, 0, st, a);        \
    else if (a.d * (int64_t)sizeof(T) % 128 != 0)                                                          \
      hipLaunchKernelGGL((layer_norm_kernel<T, NT, C, true, false, NORM>), grid, block, 0, st, a);         \
    else                                                                                                   \
      hipLaunchKernelGGL((layer_norm_kernel<T, NT, C, true, true, NORM>), grid, block, 0, st, a);          \
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
  hipLaunchKernelGGL((layer_norm_long_kernel<T, NORM>), dim3(grid_of(a.T, 1024)), dim3(1024), 0, st, a);
  return hipGetLastError();
}

template <bool NORM>
hipError_t launch_rows(const LayerNormArgs& a, int dtype, hipStream_t st) {
  switch (dtype) {
    case 0: return launch_fwd<bf16_t, NORM>(a, st);
    case 2: return launch_fwd<f16_t, NORM>(a, st);
    default: return launch_fwd<float, NORM>(a, st);
  }
}

}  // namespace

}  // namespace dora
