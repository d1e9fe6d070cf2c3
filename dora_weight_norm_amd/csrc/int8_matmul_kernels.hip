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
//
// Large products are bound by the power of the matrix cores: the bare product
// takes 351 us at 8192^3 on zeros (3.1 POP/s) and 449 on normally distributed
// rows (2.4; four waves of 128 x 128 sums 474). Measured: 8192 x 8192 x 8192 with
// r = 384, a residual and two bf16 outputs 531 to 543 us (the vendor's bare int8
// product 546); 8192 x 28672 x 8192 1.54 ms, 1.60 with GELU (2.4 POP/s).
#include "matmul_device.h"

namespace dora {

namespace {

// ---------------------------------------------------------------------------
// Up to 16 tokens and a depth of at most 8192: one workgroup a compute unit
// walks blocks of 16 columns (rows of w). Its eight waves own an eighth of the
// depth each, and the tokens' share of it stays in a wave's registers, so that
// w alone is read while it walks, and of w 64 to 128 KiB a unit are always on
// their way. (A workgroup for each block, as the
// few-rows kernel has it, spends a memory latency and two barriers beside a
// stream of 2 us, and reads the tokens from L2 for each.) Operands lie as in
// the few-rows kernel: a load takes 128 bytes of each of eight rows, and the
// two diagonal 8 x 8 blocks of a 16 x 16 product are wanted.
// The waves' sums, the pair's apart, meet in LDS, in one of two buffers, so that
// a block takes one barrier. Bound by w's bytes: 16 x 28672 x 8192 with r = 384
// 45 us (258 MB, 5.7 TB/s), 66 in the few-rows kernel.
// ---------------------------------------------------------------------------
constexpr int kWalkSteps = 8;   // of 128 bytes, a wave's share of the depth

template <typename O, int TF, bool PAIR>
__global__ __launch_bounds__(512, 1) void int8_walk_kernel(GemmArgs g, int blocks) {
  using TP = typename PairType<int8x_t, O>::type;
  constexpr int R = 2, S = kWalkSteps, SUMS = R * TF * 256;
  extern __shared__ __align__(16) float sums[];   // [2 buffers][main, pair][8 waves][SUMS]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i8 = lane & 7, chunk = lane >> 3;
  const int steps = (int)(g.K / 128), s0 = steps * wave / 8, ns = steps * (wave + 1) / 8 - s0;
  // A wave takes one step of the pair, whose rows are whole chunks; past them zeros.
  const bool in_pair = wave * 128 + chunk * 16 < g.K2 * 2;
  auto pair_chunk = [&](const char* row) __attribute__((always_inline)) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (in_pair) v = *reinterpret_cast<const u32x4_any*>(row + wave * 128 + chunk * 16);
    return v;
  };
  u32x4 x[S][TF], tp[TF];
#pragma unroll
  for (int t = 0; t < TF; ++t) {
    const int64_t m = t * 8 + i8 < g.M ? t * 8 + i8 : g.M - 1;   // (tokens past the end are not stored)
    const char* p = static_cast<const char*>(g.a) + m * g.lda + s0 * 128 + chunk * 16;
#pragma unroll
    for (int i = 0; i < S; ++i)
      if (i < ns) x[i][t] = *reinterpret_cast<const u32x4_any*>(p + i * 128);
    if constexpr (PAIR)
      tp[t] = pair_chunk(static_cast<const char*>(g.a2) + m * g.lda2 * 2);
  }
  // A block's rows of w: when one half is multiplied, its registers take the
  // next block's.
  u32x4 w[S][R], b[R];
  auto load = [&](int blk, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t c = (int64_t)blk * (8 * R) + r * 8 + i8, n = c < g.N ? c : g.N - 1;
      const char* p = static_cast<const char*>(g.b) + n * g.ldb + s0 * 128 + chunk * 16;
#pragma unroll
      for (int i = half * (S / 2); i < (half + 1) * (S / 2); ++i)
        if (i < ns) w[i][r] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p + i * 128));
      if (PAIR && half == 1) b[r] = pair_chunk(static_cast<const char*>(g.b2) + n * g.ldb2 * 2);
    }
  };
  const int step = gridDim.x;
  int blk = blockIdx.x, par = 0;
  if (blk >= blocks) return;
  load(blk, 0);
  load(blk, 1);
  for (; blk < blocks; blk += step, par ^= 1) {   // (uniform)
    float* to = sums + par * (PAIR ? 2 : 1) * 8 * SUMS;
    float* at = to + wave * SUMS + lane * 4;
    f32x4 acc[R][TF];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TF; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = half * (S / 2); i < (half + 1) * (S / 2); ++i)
        if (i < ns) {
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int t = 0; t < TF; ++t) acc[r][t] = Op16<int8x_t>::run(&w[i][r], &x[i][t], acc[r][t]);
        }
      if (PAIR && half == 1) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int t = 0; t < TF; ++t)
            *reinterpret_cast<f32x4*>(at + 8 * SUMS + (r * TF + t) * 256) =
                Op16<TP>::run(&b[r], &tp[t], f32x4{0.f, 0.f, 0.f, 0.f});
      }
      if (blk + step < blocks) load(blk + step, half);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TF; ++t)
        *reinterpret_cast<f32x4*>(at + (r * TF + t) * 256) =
            __builtin_convertvector(__builtin_bit_cast(i32x4, acc[r][t]), f32x4);
    __syncthreads();
    if (threadIdx.x < 64 * R * TF) {
      const int nl = threadIdx.x % (8 * R), m = threadIdx.x / (8 * R);
      const int64_t n = (int64_t)blk * (8 * R) + nl;
      if (m < g.M && n < g.N) {
        // (sum (i, j) of a 16 x 16 block is value i % 4 of lane 16 (i / 4) + j)
        const float* from = to + ((nl / 8) * TF + m / 8) * 256 + (16 * ((nl % 8) / 4) + m % 8) * 4 + nl % 4;
        constexpr int kOther = (16 * 2 + 8) * 4;   // from sum (i, j) to sum (i + 8, j + 8)
        float v = 0.f, p = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
          v += from[w * SUMS] + from[w * SUMS + kOther];
          if constexpr (PAIR) p += from[(8 + w) * SUMS] + from[(8 + w) * SUMS + kOther];
        }
        v = v * g.pair_rows[m] * g.w_scale[n];
        if constexpr (PAIR) v = fmaf(g.s, p, v);
        const float cs = g.ep.col_scale ? g.ep.col_scale[n] : 1.f, bs = g.ep.bias ? g.ep.bias[n] : 0.f;
        epilogue1<O>(g.ep, v, cs, bs, m, (int64_t)m * g.N + n);
      }
    }
  }
}

template <typename O, int TF, bool PAIR>
hipError_t launch_walk(GemmArgs g, hipStream_t st) {
  const int blocks = (int)((g.N + 15) / 16);
  constexpr int lds = 2 * (PAIR ? 2 : 1) * 8 * 2 * TF * 256 * 4;
  auto k = int8_walk_kernel<O, TF, PAIR>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k, dim3((unsigned)(blocks < 256 ? blocks : 256)), dim3(512), lds, st, g, blocks);
  return hipGetLastError();
}

template <typename O, int TF>
hipError_t launch_walk_any(GemmArgs g, hipStream_t st) {
  if constexpr (sizeof(O) == 2) {
    if (g.K2 > 0) return launch_walk<O, TF, true>(g, st);
  }
  return launch_walk<O, TF, false>(g, st);
}

template <typename O>
hipError_t launch(GemmArgs g, int cfg, hipStream_t st) {
  if (cfg == kWalk8) return launch_walk_any<O, 1>(g, st);
  if (cfg == kWalk16) return launch_walk_any<O, 2>(g, st);
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
