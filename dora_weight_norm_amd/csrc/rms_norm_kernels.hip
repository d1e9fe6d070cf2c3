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
#include "dora_device.h"
#include "dora_launch.h"

namespace dora {

namespace {

constexpr float kE4m3Max = 448.f;
// Inputs of more than this stream past the caches, which they would only
// empty: measured at 8192 x 8192 bf16 to 8 bits 84 us with ordinary loads and
// stores, 77.5 us with non-temporal ones; at 777 x 3583, which the caches
// hold, 8.1 and 8.6 us. Loads only where rows are whole 128-byte lines: two
// rows share a line otherwise, which was then read twice (5568 x 3000: 27.2 us
// with both, 22.6 with the stores alone). The backward's loads by the same rule,
// its stores through the caches (9000 x 1000 bf16: 48.8 us with non-temporal
// loads, 38.1 without; 2200 x 4100 38.4, 30.0; 5568 x 3000 43.6, 45.0).
constexpr int64_t kStreamBytes = (int64_t)16 << 20;
constexpr int64_t kFwdGrid = 1024;   // workgroups of 256 threads, four a compute unit
// Smallest scale: rows whose largest |n| is below 448 times it (about 2^-91)
// keep it, so that the reciprocal stays finite.
constexpr float kMinScale = 0x1p-100f;

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// One 16-byte chunk of a row: elements [k, k + E), zeros past d. STREAM: the
// rows pass the caches by (see kStreamBytes).
template <typename T, bool STREAM = false>
__device__ __forceinline__ u32x4 load_row_chunk(const T* row, int64_t k, int64_t d) {
  constexpr int E = Elem<T>::epc;
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k + E <= d) {
    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row + k);
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    return *p;
  }
  if (k < d) {
    T tmp[E];
#pragma unroll
    for (int e = 0; e < E; ++e) tmp[e] = (k + e < d) ? row[k + e] : T(0);
    __builtin_memcpy(&v, tmp, 16);
  }
  return v;
}

template <typename T, bool STREAM = false>
__device__ __forceinline__ void store_row_chunk(T* row, int64_t k, int64_t d, const float (&f)[Elem<T>::epc]) {
  constexpr int E = Elem<T>::epc;
  if (k + E <= d) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(pack<T, E>(f), reinterpret_cast<u32x4_any*>(row + k));
    else
      *reinterpret_cast<u32x4_any*>(row + k) = pack<T, E>(f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < d) row[k + e] = from_f32<T>(f[e]);
  }
}

// E fp32 values to e4m3 (OCP, round to nearest even), four to a word.
template <int E, bool STREAM = false>
__device__ __forceinline__ void store_row_q(uint8_t* row, int64_t k, int64_t d, const float (&f)[E]) {
  uint32_t w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i], f[4 * i + 1], 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * i + 2], f[4 * i + 3], v, true);
    w[i] = (uint32_t)v;
  }
  if (k + E <= d) {
    if constexpr (E == 8) {
      const u32x2 p = {w[0], w[1]};
      if constexpr (STREAM)
        __builtin_nontemporal_store(p, reinterpret_cast<u32x2_any*>(row + k));
      else
        *reinterpret_cast<u32x2_any*>(row + k) = p;
    } else {
      *reinterpret_cast<u32_any*>(row + k) = w[0];
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < d) row[k + e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

// E weights (fp32) of a chunk; ones where there are none, zeros past d.
template <int E>
__device__ __forceinline__ void load_weight(const float* w, int64_t k, int64_t d, float (&f)[E]) {
  if (w == nullptr) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = 1.f;
  } else if (k + E <= d) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const u32x4 v = *reinterpret_cast<const u32x4_any*>(w + k + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * i + e] = __uint_as_float(v[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = (k + e < d) ? w[k + e] : 0.f;
  }
}

// Sum over the NT threads that share a row, in a fixed order: inside each
// wave by lane exchanges, then over the waves in increasing order. `slot`
// names the LDS words used, a different one for each call before a barrier.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v += lds[i];
  }
  return v;
}

// Largest |value| over the row, carried as its bits: among non-negative
// floats the order of the bits is the order of the values, and a NaN's bits
// are above infinity's, so a NaN anywhere comes out as a NaN.
template <int NT>
__device__ __forceinline__ uint32_t row_max_bits(uint32_t v, uint32_t* lds) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, m, 64);
    v = o > v ? o : v;
  }
  if constexpr (NT > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v = lds[i] > v ? lds[i] : v;
  }
  return v;
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// scale = top / 448: 1 for a row of zeros, at least kMinScale otherwise; NaN
// or infinite where top is.
__device__ __forceinline__ float scale_of(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits);
  const float s = top / kE4m3Max;
  return top_bits == 0 ? 1.f : (s < kMinScale ? kMinScale : s);
}

// The quotient n / scale, correctly rounded in fp32 without a division a value:
// n times the rounded reciprocal is within a step of it, and adding the exact
// remainder times the reciprocal gives the nearest value (Markstein 1990). The
// product alone put values beside the border of two 8-bit steps on the wrong
// side of it; the two operations more cost 0.7 us of 78 at 8192 x 8192. An
// infinite scale leaves 0 (NaN where n is infinite), as the division does.
struct RowQuotient {
  float inv, s;
  __device__ __forceinline__ explicit RowQuotient(float scale)
      : inv(1.f / scale), s(scale <= 3.402823466e38f ? scale : 0.f) {}
  __device__ __forceinline__ float operator()(float n) const {
    const float q = n * inv;
    return fmaf(fmaf(-q, s, n), inv, q);
  }
};

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

// out0[j] (j < n0) or out1[j - n0] = sum of column j over the n_part rows of
// part [n_part][n]; either output may be null. One workgroup owns 64 columns;
// its sixteen waves each add a contiguous sixteenth of the rows in increasing
// order (loads kSumBatch at a time), then wave 0 adds those sums in order.
constexpr int kSumCols = 64, kSumSplit = 16, kSumBatch = 16;

__global__ __launch_bounds__(kSumCols* kSumSplit) void column_sum_kernel(const float* part, int n_part, int64_t n,
                                                                          float* out0, int64_t n0, float* out1) {
  __shared__ float red[kSumSplit][kSumCols];
  const int c = threadIdx.x % kSumCols, q = threadIdx.x / kSumCols;
  const int64_t j = (int64_t)blockIdx.x * kSumCols + c;
  const int y0 = (int)((int64_t)n_part * q / kSumSplit), y1 = (int)((int64_t)n_part * (q + 1) / kSumSplit);
  float acc = 0.f;
  if (j < n) {
    const float* col = part + j;
    int y = y0;
    for (; y + kSumBatch <= y1; y += kSumBatch) {
      float v[kSumBatch];
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) v[u] = col[(int64_t)(y + u) * n];
#pragma unroll
      for (int u = 0; u < kSumBatch; ++u) acc += v[u];
    }
    for (; y < y1; ++y) acc += col[(int64_t)y * n];
  }
  red[q][c] = acc;
  __syncthreads();
  if (q != 0 || j >= n) return;
#pragma unroll
  for (int k = 1; k < kSumSplit; ++k) acc += red[k][c];
  if (j < n0) {
    if (out0) out0[j] = acc;
  } else if (out1) {
    out1[j - n0] = acc;
  }
}

// Threads and chunks a thread that hold a row of d elements; nt 0: too long.
struct RowShape {
  int nt, c;
};

// Forward. Many short rows take a wave each (no barrier; 5568 x 1000: 10.8 us,
// 15.9 with 256 threads a row), up to two chunks a thread; other rows take 256
// threads (5568 x 1456: 16.8 us, 19.2 with a wave of four chunks a thread), 512 past two chunks a thread (four of 8192 bf16 elements ran
// two workgroups a compute unit for their registers: 80 against 77.5 us), or
// 1024 where there are too few rows to fill the chip. Rows of up to 16384 elements stay in registers
// (1024 threads have 128 registers each: two 16-bit chunks or four fp32).
RowShape forward_shape(int64_t T, int64_t d, int epc) {
  const int64_t ch = (d + epc - 1) / epc;
  auto fit = [&](int nt) {
    const int64_t c = (ch + nt - 1) / nt;
    return (int)(c <= 1 ? 1 : (c <= 2 ? 2 : (c <= 4 ? 4 : (c <= 8 ? 8 : 0))));
  };
  if (ch <= 128 && (T >= 512 || ch <= 64)) return RowShape{64, fit(64)};
  if (ch <= 512 && (T >= 512 || ch <= 256)) return RowShape{256, fit(256)};
  if (ch <= 2048 && T >= 512) return RowShape{512, fit(512)};
  return ch <= (epc == 8 ? 2048 : 4096) ? RowShape{1024, fit(1024)} : RowShape{0, 0};
}

// Backward: workgroups of 64 to 512 threads, at most four chunks a thread
// (weights and sums are held beside them).
RowShape backward_shape(int64_t d, int epc) {
  const int64_t ch = (d + epc - 1) / epc;
  if (ch <= 64) return RowShape{64, 1};
  if (ch <= 256) return RowShape{256, 1};
  if (ch <= 512) return RowShape{256, 2};
  if (ch <= 1024) return RowShape{512, 2};
  return ch <= 2048 ? RowShape{512, 4} : RowShape{0, 0};
}

// Workgroups of the backward: enough waves to fill the chip (256 compute
// units), few enough that the dweight partials stay small beside the rows.
int64_t backward_grid(int64_t T, int64_t d, int epc) {
  const RowShape r = backward_shape(d, epc);
  const int64_t g = r.nt == 64 ? 2048 : (r.nt == 256 ? 512 : 256);
  return T < g ? T : g;
}

// Workgroups of the forward: one a row (or four rows), up to what the chip
// holds at once; past that each takes several rows.
unsigned grid_of(int64_t n, int nt) {
  const int64_t most = nt == 1024 ? 512 : kFwdGrid;
  return (unsigned)(n < most ? n : most);
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
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((n + kSumCols - 1) / kSumCols)), dim3(kSumCols * kSumSplit), 0,
                     st, part, n_part, n, out0, n0, out1);
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
