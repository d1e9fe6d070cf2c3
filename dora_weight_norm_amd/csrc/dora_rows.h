// Rows of a norm or a quantiser: loads and stores of any length and alignment,
// sums and maxima over a row, 8-bit scales, and how many threads a row takes.
#pragma once

#include "dora_device.h"

namespace dora {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kInt8Max = 127.f;
enum : int { kQE4m3 = 0, kQInt8 = 1 };   // what 8-bit rows hold
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

// E bytes of a row chunk, four to a word.
template <int E, bool STREAM = false>
__device__ __forceinline__ void store_row_bytes(uint8_t* row, int64_t k, int64_t d, const uint32_t (&w)[E / 4]) {
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

// E bytes of a row from column k on, zeros past d.
template <int E, bool STREAM = false>
__device__ __forceinline__ void load_row_bytes(const uint8_t* row, int64_t k, int64_t d, uint32_t (&w)[E / 4]) {
  if (k + E <= d) {
    if constexpr (E == 8) {
      const u32x2_any* p = reinterpret_cast<const u32x2_any*>(row + k);
      u32x2 v;
      if constexpr (STREAM)
        v = __builtin_nontemporal_load(p);
      else
        v = *p;
      w[0] = v[0], w[1] = v[1];
    } else {
      w[0] = *reinterpret_cast<const u32_any*>(row + k);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) w[i] = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < d) w[e / 4] |= (uint32_t)row[k + e] << (8 * (e % 4));
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
  store_row_bytes<E, STREAM>(row, k, d, w);
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

// Sum over the wave, the same in every lane: over quads and rows of 16 by lane
// permutes of the vector unit (a few cycles each, where a shuffle goes through
// LDS), then over the four rows.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

__device__ __forceinline__ float lane_of(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

__device__ __forceinline__ float row16_sum(float v) {   // over each row of 16 lanes
  v += dpp<0xb1>(v);    // lane ^ 1
  v += dpp<0x4e>(v);    // lane ^ 2
  v += dpp<0x141>(v);   // mirror of eight
  v += dpp<0x140>(v);   // mirror of sixteen
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  return (lane_of(v, 0) + lane_of(v, 16)) + (lane_of(v, 32) + lane_of(v, 48));
}

__device__ __forceinline__ uint32_t row16_max(uint32_t u) {
  auto step = [&](uint32_t o) __attribute__((always_inline)) { u = o > u ? o : u; };
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0xb1, 0xf, 0xf, true));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x4e, 0xf, 0xf, true));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x141, 0xf, 0xf, true));
  step((uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, 0x140, 0xf, 0xf, true));
  return u;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t u) {
  u = row16_max(u);
  uint32_t m = (uint32_t)__builtin_amdgcn_readlane((int)u, 0);
#pragma unroll
  for (int i = 16; i < 64; i += 16) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)u, i);
    m = o > m ? o : m;
  }
  return m;
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

// The scale of integers, max |x| / 127 correctly rounded in fp32: the product with
// the rounded reciprocal and its exact remainder's share, as in RowQuotient (equal
// to the division for every fp32 maximum from 2^-93 on; the product alone is a
// step off for one in forty of them, among them six of the 128 significands of
// bf16, where half of the maximum then came out as 64 instead of 63). 1 for a row
// of zeros, at least kMinScale otherwise, NaN or infinite where the largest value is.
__device__ __forceinline__ float int8_scale_of(uint32_t top_bits) {
  constexpr float kInv = 1.f / kInt8Max;
  const float top = __uint_as_float(top_bits), q = top * kInv;
  const float s = top_bits < 0x7f800000u ? fmaf(fmaf(-q, kInt8Max, top), kInv, q) : q;
  return top_bits == 0 ? 1.f : (s < kMinScale ? kMinScale : s);
}

// The integer nearest to n / scale (to the quotient itself, not to one rounded
// in fp32), ties to the even one, in the low byte of the result: three 64-bit
// operations a value. The reciprocal is good to 2^-45 and the quotient rounded
// to steps of 2^-30, on which a tie lies and from which no other quotient of
// two fp32 numbers is nearer to a tie than 2^-26; then to whole steps. NaN (of
// rows with a NaN or an infinity) gives 0: its low bits are 0. Rows of few
// significant bits meet ties often (half of the largest value is 63.5 steps),
// and a quotient rounded in fp32 took them to either side. The same by an fp32
// quotient, its remainder and a comparison took seventeen operations a value,
// as long as the memory (8192 x 8192 bf16 in groups of 128).
struct WholeSteps {
  double inv;
  __device__ __forceinline__ explicit WholeSteps(float scale) {
    const double s = scale, r = __builtin_amdgcn_rcpf(scale);
    inv = fma(r, fma(-s, r, 1.0), r);
    if (!(scale <= 3.402823466e38f)) inv = __builtin_nan("");
  }
  __device__ __forceinline__ uint32_t operator()(float n) const {
    constexpr double kFine = 0x1.8p22, kWhole = 0x1.8p52;
    const double v = fma((double)n, inv, kFine) + (kWhole - kFine);
    return (uint32_t)__builtin_bit_cast(uint64_t, v);
  }
};

// The low bytes of E words.
template <int E>
__device__ __forceinline__ void low_bytes(const uint32_t (&v)[E], uint32_t (&w)[E / 4]) {
#pragma unroll
  for (int i = 0; i < E / 4; ++i)   // (of two words each, then the two halves)
    w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(v[4 * i + 3], v[4 * i + 2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(v[4 * i + 1], v[4 * i], 0x0c0c0400u), 0x05040100u);
}

// E fp32 values of a row chunk as 8-bit integers.
template <int E, bool STREAM = false>
__device__ __forceinline__ void store_row_int8(uint8_t* row, int64_t k, int64_t d, const float (&f)[E],
                                               const WholeSteps& steps) {
  uint32_t v[E], w[E / 4];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = steps(f[e]);
  low_bytes<E>(v, w);
  store_row_bytes<E, STREAM>(row, k, d, w);
}

// C chunks of a row, NT threads apart, in the 8-bit type that `kind` names,
// with the scale of the row's largest |value|, which it returns.
template <int E, int NT, int C, bool STREAM>
__device__ __forceinline__ float store_row_8(uint8_t* row, int lane, int64_t d, const float (&f)[C][E], uint32_t top,
                                             int kind) {
  if (kind == kQInt8) {
    const float s = int8_scale_of(top);
    const WholeSteps steps(s);
#pragma unroll
    for (int c = 0; c < C; ++c) store_row_int8<E, STREAM>(row, (int64_t)(c * NT + lane) * E, d, f[c], steps);
    return s;
  }
  const float s = scale_of(top);
  const RowQuotient quotient(s);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = quotient(f[c][e]);
    store_row_q<E, STREAM>(row, (int64_t)(c * NT + lane) * E, d, v);
  }
  return s;
}

// out0[j] (j < n0) or out1[j - n0] = sum of column j over the n_part rows of
// part [n_part][n]; either output may be null. One workgroup owns 64 columns;
// its sixteen waves each add a contiguous sixteenth of the rows in increasing
// order (loads kSumBatch at a time), then wave 0 adds those sums in order.
constexpr int kSumCols = 64, kSumSplit = 16, kSumBatch = 16, kSumThreads = kSumCols * kSumSplit;
struct ColumnSum {
  const float* part;
  int n_part;
  int64_t n;
  float* out0;
  int64_t n0;
  float* out1;
};
[[maybe_unused]] unsigned sum_groups(int64_t n) { return (unsigned)((n + kSumCols - 1) / kSumCols); }

__device__ __forceinline__ void column_sum(const ColumnSum& s, unsigned block) {
  __shared__ float red[kSumSplit][kSumCols];
  const int c = threadIdx.x % kSumCols, q = threadIdx.x / kSumCols;
  const int64_t j = (int64_t)block * kSumCols + c, n = s.n;
  const int y0 = (int)((int64_t)s.n_part * q / kSumSplit), y1 = (int)((int64_t)s.n_part * (q + 1) / kSumSplit);
  float acc = 0.f;
  if (j < n) {
    const float* col = s.part + j;
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
  if (j < s.n0) {
    if (s.out0) s.out0[j] = acc;
  } else if (s.out1) {
    s.out1[j - s.n0] = acc;
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
[[maybe_unused]] RowShape forward_shape(int64_t T, int64_t d, int epc) {
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
[[maybe_unused]] int64_t backward_grid(int64_t T, int64_t d, int epc) {
  const RowShape r = backward_shape(d, epc);
  const int64_t g = r.nt == 64 ? 2048 : (r.nt == 256 ? 512 : 256);
  return T < g ? T : g;
}

// Workgroups of the forward: one a row (or four rows), up to what the chip
// holds at once; past that each takes several rows.
[[maybe_unused]] unsigned grid_of(int64_t n, int nt) {
  const int64_t most = nt == 1024 ? 512 : kFwdGrid;
  return (unsigned)(n < most ? n : most);
}

}  // namespace

}  // namespace dora
