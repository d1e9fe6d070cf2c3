// A scale of int8 rows as a power of two and a factor, for products of 16-bit operands.
#pragma once

#include "dora_device.h"

namespace dora {

namespace {

// scale = power (FoldBits) * fold_factor. An integer of 8 bits times the power is exact in T
// and finite: it is between 2^-24 and 2^8 for fp16 (128 2^8 is in its range), 2^-126 and
// 2^120 for bf16. So one scale a row, which runs along a product's depth, costs its rows
// no rounding when the other operand holds the factor, whose own rounding takes it in.
// Inside those limits the factor is between a half and 1 (of fp16 rows of more than 2^15
// up to 2.02, where a gradient that passes the range leaves it in the result too). The
// factor of 0, of an infinity and of NaN is that itself.
//
// On the bits, without a branch for a loop that may or may not fold: (scale and mask) +
// add, between low and high; all of them idle where nothing is folded.
template <typename T>
struct FoldBits {
  uint32_t mask, add, low, high;
  __device__ __forceinline__ explicit FoldBits(bool fold) {
    constexpr bool kHalf = std::is_same<T, f16_t>::value;
    mask = fold ? 0x7f800000u : ~0u;
    add = fold ? 0x00800000u : 0u;
    low = fold && kHalf ? 0x33800000u : 0u;
    high = fold ? (kHalf ? 0x43800000u : 0x7b800000u) : ~0u;
  }
  __device__ __forceinline__ float operator()(float scale) const {
    uint32_t p = (__float_as_uint(scale) & mask) + add;
    p = p < high ? p : high;
    return __uint_as_float(p > low ? p : low);
  }
};

template <typename T>
__device__ __forceinline__ float fold_factor(float scale) {
  // (times the power's reciprocal, whose exponent is 254 less the power's)
  return scale * __uint_as_float(0x7f000000u - __float_as_uint(FoldBits<T>(true)(scale)));
}

}  // namespace

}  // namespace dora
