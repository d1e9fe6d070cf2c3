// The backward's products with one operand held as int8 rows, which the tile
// kernel (matmul_device.h) brings to 16 bits on its way to LDS:
//
//   dx = du (scale q_w)       dw = du^T (scale q_x)
//
// The 256-row tile has eight waves, as for 16-bit operands, each of which converts
// an eighth of a stage, two values between two of its matrix instructions, under
// those of the other wave of its SIMD. Four waves of 128 x 128 sums took as long
// where the depth is short and 5% longer at 8192^3 (dx 990 us, 942 so). Measured:
// dw of 8192 x 384 x 8192 with x in groups of 128 columns 89 us, the element-wise
// pass and the joining of four parts in it; 4096^3 142 us, as from 16-bit copies.
#include "matmul_device.h"

namespace dora {

namespace {

template <typename T, bool AT>
hipError_t launch(GemmArgs g, int cfg, hipStream_t st) {
  split_stages(g, 64, 64);
  hipError_t e = hipErrorInvalidValue;
  if (cfg == kTile256) e = launch_tile<T, T, 2, 4, 4, 2, 2, false, AT, true, true>(g, st);
  if (cfg == kTile128) e = launch_tile<T, T, 2, 2, 2, 2, 2, false, AT, true, true>(g, st);
  return e != hipSuccess || g.splits == 1 ? e : launch_join<T>(g, st);
}

}  // namespace

hipError_t gemm_rows8(const GemmArgs& g, int dtype, bool a_across, int cfg, hipStream_t st) {
  if (dtype == 0) return a_across ? launch<bf16_t, true>(g, cfg, st) : launch<bf16_t, false>(g, cfg, st);
  return a_across ? launch<f16_t, true>(g, cfg, st) : launch<f16_t, false>(g, cfg, st);
}

}  // namespace dora
