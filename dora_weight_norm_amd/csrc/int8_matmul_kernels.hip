// Matrix product in 8-bit integers with scales for each token and channel:
//
//   u = row_scale[m] w_scale[n] sum_k x[m,k] w[n,k] + s sum_l t[m,l] b[n,l]
//   y = act(col_scale[n] u + bias[n]) + residual[m,n]
//
// on the kernels of the other products (matmul_device.h). The integer sums are
// exact: int32 on the matrix cores, at the rate of the 8-bit floating ones. A
// workgroup converts and scales its sums in the registers; the pair, bf16 or
// fp16 like the outputs, then runs through the same accumulators, which hold
// the main sums divided by s and are multiplied by it at the end, so that s
// costs no rounding of an operand.
#include "matmul_device.h"

namespace dora {

namespace {

template <typename O>
hipError_t launch(GemmArgs g, int cfg, hipStream_t st) {
  if (cfg == kFew8) return launch_few_rows<int8x_t, O, 2, 1>(g, st);
  if (cfg == kFew16) return launch_few_rows<int8x_t, O, 2, 2>(g, st);
  if (cfg == kFew32) return launch_few_rows<int8x_t, O, 4, 4>(g, st);
  split_stages(g, 128, 64);
  hipError_t e = hipErrorInvalidValue;
  if (g.K2 > 0) {
    if constexpr (sizeof(O) == 2) {
      if (cfg == kTile256) e = launch_tile<int8x_t, O, 2, 4, 4, 2, 2, true>(g, st);
      if (cfg == kTile128) e = launch_tile<int8x_t, O, 2, 2, 2, 2, 2, true>(g, st);
      if (cfg == kTile64) e = launch_tile<int8x_t, O, 2, 2, 1, 1, 4, true>(g, st);
    }
  } else {
    if (cfg == kTile256) e = launch_tile<int8x_t, O, 2, 4, 4, 2, 2, false>(g, st);
    if (cfg == kTile128) e = launch_tile<int8x_t, O, 2, 2, 2, 2, 2, false>(g, st);
    if (cfg == kTile64) e = launch_tile<int8x_t, O, 2, 2, 1, 1, 4, false>(g, st);
  }
  return e != hipSuccess || g.splits == 1 ? e : launch_join<O>(g, st);
}

}  // namespace

hipError_t gemm_int8(const GemmArgs& g, int out_dtype, int cfg, hipStream_t st) {
  switch (out_dtype) {
    case 0: return launch<bf16_t>(g, cfg, st);
    case 2: return launch<f16_t>(g, cfg, st);
    default: return launch<float>(g, cfg, st);
  }
}

}  // namespace dora
