// Rows in 8-bit integers on gfx950: groups of columns packed with one scale
// each, and packed rows back in a storage type (whole rows are packed by the
// layer norm's kernel without its norm).
//
//   scale = max |x| / 127 over a group      q = x / scale to the nearest integer
//   x = q * scale
//
// HBM bound: 3.03 bytes an element of 16 bits in groups of 128. A thread takes
// 16 bytes of a row, so a group is 4 to 64 lanes of one wave and its maximum a
// few lane exchanges: no LDS, no barrier. Measured, 8192 x 8192 bf16 in groups
// of 128: packing 37 to 38 us (5.4 TB/s), back 34 us (5.9 TB/s).
#include "layer_norm_device.h"

namespace dora {

namespace {

// A workgroup of 256 threads is `bx` threads along a row by 256 / bx rows; an
// item is one such step, `steps` of them along a row. kItems items' loads are
// in flight at a time.
constexpr int kItems = 2;
constexpr int64_t kMostGroups = 65536;   // workgroups

struct RowSteps {
  int64_t T, d;
  int64_t groups;      // scales a row
  int shift;           // log2 of the columns of a group (group_shift)
  uint32_t steps, items;
};

struct Place {
  int64_t row, k;      // row, and first column
  bool ok;
};

template <int E>
__device__ __forceinline__ Place place_of(const RowSteps& s, uint32_t item) {
  const uint32_t r = item / s.steps, c = item - r * s.steps;   // (uniform)
  Place p;
  p.row = (int64_t)r * blockDim.y + threadIdx.y;
  p.k = ((int64_t)c * blockDim.x + threadIdx.x) * E;
  p.ok = item < s.items && p.row < s.T && p.k < s.d;
  return p;
}

template <typename T, int L, bool STREAM>
__global__ __launch_bounds__(256) void quantize_groups_kernel(const T* x, RowSteps s, uint8_t* q, float* scale) {
  constexpr int E = Elem<T>::epc;
  for (uint32_t it = blockIdx.x * kItems; it < s.items; it += gridDim.x * kItems) {   // (uniform)
    u32x4 v[kItems];
    Place p[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      p[i] = place_of<E>(s, it + i);
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (p[i].ok) v[i] = load_row_chunk<T, STREAM>(x + p[i].row * s.d, p[i].k, s.d);
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      float f[E];
      unpack<T, E>(v[i], f);
      uint32_t top = 0;   // (past d the values are zeros)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t b = abs_bits(f[e]);
        top = b > top ? b : top;
      }
#pragma unroll
      for (int m = L / 2; m >= 1; m >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, m, 64);
        top = o > top ? o : top;
      }
      const float sc = int8_scale_of(top);
      const WholeSteps steps(sc);
      if (p[i].ok) {
        if (threadIdx.x % L == 0) scale[p[i].row * s.groups + (p[i].k >> s.shift)] = sc;
        store_row_int8<E, STREAM>(q + p[i].row * s.d, p[i].k, s.d, f, steps);
      }
    }
  }
}

// One or two operands of rows of d columns, the second's rows numbered after the
// first's; rows of x lie ld >= d elements apart, and those from d on, up to a
// whole chunk or ld, are written as zeros.
struct UnpackJob {
  const uint8_t* q;
  const float* scale;
  int64_t groups, T;
  int shift;
  void* x;
};

template <typename T, bool STREAM>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(UnpackJob a, UnpackJob b, RowSteps s, int64_t ld) {
  constexpr int E = Elem<T>::epc;
  for (uint32_t it = blockIdx.x * kItems; it < s.items; it += gridDim.x * kItems) {
    uint32_t w[kItems][E / 4];
    float sc[kItems];
    Place p[kItems];
    T* to[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      p[i] = place_of<E>(s, it + i);
      const bool first = p[i].row < a.T;
      const int64_t row = first ? p[i].row : p[i].row - a.T;
      to[i] = static_cast<T*>(first ? a.x : b.x) + row * ld;
      if (p[i].ok) {
        load_row_bytes<E>((first ? a.q : b.q) + row * s.d, p[i].k, s.d, w[i]);
        sc[i] = (first ? a.scale : b.scale)[row * (first ? a.groups : b.groups) + (p[i].k >> (first ? a.shift : b.shift))];
      }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (!p[i].ok) continue;
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = (float)(int8_t)(w[i][e / 4] >> (8 * (e % 4))) * sc[i];
      store_row_chunk<T, STREAM>(to[i], p[i].k, ld, f);
    }
  }
}

int log2_of(int64_t v) {
  int s = 0;
  while (((int64_t)1 << s) < v) ++s;
  return s;
}

// The steps of rows whose chunks of E elements are padded to whole groups of L.
RowSteps row_steps(int64_t T, int64_t d, int64_t group, int E, int L, dim3* grid, dim3* block) {
  RowSteps s{};
  s.T = T, s.d = d;
  s.groups = scales_of(d, group);
  s.shift = group_shift(group);
  const int64_t chunks = ((d + E - 1) / E + L - 1) / L * L;
  int64_t bx = (int64_t)1 << log2_of(chunks);
  if (bx > 256) bx = 256;
  const int64_t by = 256 / bx;
  s.steps = (uint32_t)((chunks + bx - 1) / bx);
  s.items = (uint32_t)((T + by - 1) / by * s.steps);
  const int64_t groups = ((int64_t)s.items + kItems - 1) / kItems;
  *grid = dim3((unsigned)(groups < kMostGroups ? groups : kMostGroups));
  *block = dim3((unsigned)bx, (unsigned)by);
  return s;
}

template <typename T>
hipError_t quantize_groups(const void* x, int64_t T_, int64_t d, int64_t group, void* q, float* scale, hipStream_t st) {
  constexpr int E = Elem<T>::epc;
  const int L = (int)(group / E);
  dim3 grid, block;
  const RowSteps s = row_steps(T_, d, group, E, L, &grid, &block);
  const bool stream = T_ * d * (int64_t)sizeof(T) > kStreamBytes && d * (int64_t)sizeof(T) % 128 == 0;
#define DORA_GROUPS(LANES)                                                                                         \
  if (L == LANES) {                                                                                                \
    if (stream)                                                                                                    \
      hipLaunchKernelGGL((quantize_groups_kernel<T, LANES, true>), grid, block, 0, st, static_cast<const T*>(x), s, \
                         static_cast<uint8_t*>(q), scale);                                                         \
    else                                                                                                           \
      hipLaunchKernelGGL((quantize_groups_kernel<T, LANES, false>), grid, block, 0, st, static_cast<const T*>(x),   \
                         s, static_cast<uint8_t*>(q), scale);                                                      \
    return hipGetLastError();                                                                                      \
  }
  if constexpr (E == 8) {
    DORA_GROUPS(4)
  }
  DORA_GROUPS(8)
  DORA_GROUPS(16)
  DORA_GROUPS(32)
  if constexpr (E == 4) {
    DORA_GROUPS(64)
  }
#undef DORA_GROUPS
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t dequantize(const UnpackJob& a, const UnpackJob& b, int64_t d, int64_t ld, hipStream_t st) {
  dim3 grid, block;
  const RowSteps s = row_steps(a.T + b.T, d, 0, Elem<T>::epc, 1, &grid, &block);
  const bool stream = (a.T + b.T) * d * (int64_t)sizeof(T) > kStreamBytes && d % 128 == 0;
  if (stream)
    hipLaunchKernelGGL((dequantize_rows_kernel<T, true>), grid, block, 0, st, a, b, s, ld);
  else
    hipLaunchKernelGGL((dequantize_rows_kernel<T, false>), grid, block, 0, st, a, b, s, ld);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int dtype, int64_t T, int64_t d, int64_t group, void* q, float* scale,
                                hipStream_t st) {
  if (group == 0) {
    LayerNormArgs a{};
    a.x = x, a.T = T, a.d = d, a.q = q, a.q8 = kQInt8, a.scale = scale;
    return launch_rows<false>(a, dtype, st);
  }
  switch (dtype) {
    case 0: return quantize_groups<bf16_t>(x, T, d, group, q, scale, st);
    case 2: return quantize_groups<f16_t>(x, T, d, group, q, scale, st);
    default: return quantize_groups<float>(x, T, d, group, q, scale, st);
  }
}

hipError_t launch_dequantize_rows(const Int8Rows& r, int64_t T, void* x, const Int8Rows& r2, int64_t T2, void* x2,
                                  int64_t d, int64_t ld, int dtype, hipStream_t st) {
  const UnpackJob a{r.q, r.scale, scales_of(d, r.group), T, group_shift(r.group), x};
  const UnpackJob b{r2.q, r2.scale, scales_of(d, r2.group), T2, group_shift(r2.group), x2};
  switch (dtype) {
    case 0: return dequantize<bf16_t>(a, b, d, ld, st);
    case 2: return dequantize<f16_t>(a, b, d, ld, st);
    default: return dequantize<float>(a, b, d, ld, st);
  }
}

}  // namespace dora
