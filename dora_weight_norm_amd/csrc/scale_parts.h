// A scale of int8 rows as a power of two and a significand, for products of 16-bit
// operands.
#pragma once

#include "dora_device.h"

namespace dora {

namespace {

// scale = 2^fold_exp * fold_factor. An integer of 8 bits times that power is exact in
// T and finite: 128 2^8 and 2^-24 are in fp16's range. So one scale a row, which runs
// along a product's depth, costs its rows no rounding when the other operand holds the
// factor, whose own rounding takes it in. Inside those limits the factor is between a
// half and 1 (fp16 rows of more than 2^15 up to 2.02, where gradients beside them that
// pass fp16's range would leave it in the result); past them, and for 0, infinities
// and NaN (whose exponent counts as 0), it is what is left of the scale.
template <typename T>
__device__ __forceinline__ int fold_exp(float scale) {
  constexpr bool kHalf = std::is_same<T, f16_t>::value;
  constexpr int kLow = kHalf ? -24 : -126, kHigh = kHalf ? 8 : 120;
  const int e = __builtin_amdgcn_frexp_expf(scale);
  return e < kLow ? kLow : (e > kHigh ? kHigh : e);
}

template <typename T>
__device__ __forceinline__ float fold_power(float scale) {
  return ldexpf(1.f, fold_exp<T>(scale));
}

template <typename T>
__device__ __forceinline__ float fold_factor(float scale) {
  return ldexpf(scale, -fold_exp<T>(scale));
}

}  // namespace

}  // namespace dora
