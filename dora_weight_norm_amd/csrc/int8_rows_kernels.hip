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
#include "int8_rows_device.h"
#include "layer_norm_device.h"

namespace dora {

namespace {

template <typename T, int L, bool STREAM>
__global__ __launch_bounds__(256) void quantize_groups_kernel(const T* x, RowSteps s, uint8_t* q, float* scale) {
  constexpr int E = Elem<T>::epc;
  for (uint32_t it = blockIdx.x * kItems; it < s.items; it += gridDim.x * kItems) {   // (uniform)
    u32x4 v[kItems];
    Place p[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      p[i] = place_of<E>(s, it + i, threadIdx.x);
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

template <typename T, bool STREAM>
__global__ __launch_bounds__(256) void dequantize_rows_kernel(UnpackJob a, RowSteps s) {
  unpack_rows<T, STREAM, false>(a, UnpackJob{}, s, s.d, blockIdx.x, gridDim.x, threadIdx.x);
}

template <typename T>
hipError_t quantize_groups(const void* x, int64_t T_, int64_t d, int64_t group, void* q, float* scale, hipStream_t st) {
  constexpr int E = Elem<T>::epc;
  const int L = (int)(group / E);
  const RowSteps s = row_steps(T_, d, group, E, L);
  const dim3 grid(row_groups(s)), block(256);
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
hipError_t dequantize(const UnpackJob& a, int64_t d, hipStream_t st) {
  const RowSteps s = row_steps(a.T, d, 0, Elem<T>::epc, 1);
  const dim3 grid(row_groups(s)), block(256);
  if (a.T * d * (int64_t)sizeof(T) > kStreamBytes && d % 128 == 0)
    hipLaunchKernelGGL((dequantize_rows_kernel<T, true>), grid, block, 0, st, a, s);
  else
    hipLaunchKernelGGL((dequantize_rows_kernel<T, false>), grid, block, 0, st, a, s);
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

hipError_t launch_dequantize_rows(const Int8Rows& r, int64_t T, int64_t d, int dtype, void* x, hipStream_t st) {
  const UnpackJob a = unpack_job(r, T, d, x, false);
  switch (dtype) {
    case 0: return dequantize<bf16_t>(a, d, st);
    case 2: return dequantize<f16_t>(a, d, st);
    default: return dequantize<float>(a, d, st);
  }
}

}  // namespace dora
