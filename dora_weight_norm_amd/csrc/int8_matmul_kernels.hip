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
// r = 384, a residual and two bf16 outputs 528 to 547 us (the vendor's bare int8
// product 546); 8192 x 28672 x 8192 1.54 ms, 1.57 to 1.63 with GELU (2.4 POP/s).
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

// ---------------------------------------------------------------------------
// 64 x 64 of a product whose rows lie at any address: four waves of 32 x 32 sums.
// The tiles' direct loads take whole aligned chunks of 16 bytes, for which rows off
// that grid are copied first; here they go through registers, two stages of 128
// bytes ahead, the chunk at a row's end as its last 16 bytes, shifted (rows of at
// least 16 bytes). Bound by a memory latency for every two stages, which several
// workgroups a compute unit hide: four or eight stages ahead take the registers of
// theirs (64 x 8192 x 8189 22.2 us with two, 23.5 with four, 28.8 with eight). 333 x
// 1001 x 777 with r = 24: 9.7 us on the GPU, 10.7 behind copies, 11.4 and 16 with
// the host's call. The sums are scaled and joined as in the other tiles, so that an
// operand's address does not change a result.
// ---------------------------------------------------------------------------
// Sixteen bytes without the first `drop` of them, zeros behind.
__device__ __forceinline__ u32x4 dropped(u32x4 v, int drop) {
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  if (drop >= 8) lo = hi, hi = 0, drop -= 8;
  if (drop >= 8) lo = 0, drop = 0;
  if (drop > 0) lo = lo >> (8 * drop) | hi << (64 - 8 * drop), hi >>= 8 * drop;
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

template <typename O, bool PAIR>
__global__ __launch_bounds__(256) void int8_any_kernel(GemmArgs g) {
  using TP = typename PairType<int8x_t, O>::type;
  constexpr int AHEAD = 2, BUF = 128 * 128, LD = 68;   // LD: floats of an epilogue row (padded)
  __shared__ __align__(16) char lds[2 * BUF];          // [2][a's 64 rows, b's 64 rows][128]; then the sums
  static_assert(64 * LD * 4 <= 2 * BUF, "the epilogue fits");
  __shared__ __align__(16) float scales[2][64];        // with a pair: of the rows and the columns
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, fr = lane & 31, fg = lane >> 5;
  const int total = g.n_mt * g.n_nt, split = blockIdx.x / total, id = blockIdx.x - split * total;
  const int64_t m0 = (int64_t)(id % g.n_mt) * 64, n0 = (int64_t)(id / g.n_mt) * 64;
  // A thread takes chunk c of rows r and r + 32 of both operands. (Rows past the
  // end read the last one's and are not stored.)
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3;
  const char *p[4], *p2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = (i < 2 ? m0 : n0) + r + 32 * (i % 2), last = (i < 2 ? g.M : g.N) - 1, row = at < last ? at : last;
    p[i] = static_cast<const char*>(i < 2 ? g.a : g.b) + row * (i < 2 ? g.lda : g.ldb);
    p2[i] = static_cast<const char*>(i < 2 ? g.a2 : g.b2) + row * (i < 2 ? g.lda2 : g.ldb2) * 2;
  }
  const int n1 = (int)((g.K + 127) / 128), st0 = split * g.stages_per_split;
  const int st1 = st0 + g.stages_per_split < g.stages ? st0 + g.stages_per_split : g.stages;
  // Of the result a thread has eight columns of rows r and r + 32; what scales them
  // is asked for here, a depth before it is needed.
  const int64_t n = n0 + c * 8, m[2] = {m0 + r, m0 + r + 32}, off[2] = {m[0] * g.N + n, m[1] * g.N + n};
  const int nv = (int)(g.N - n < 8 ? g.N - n : 8);
  const bool ok[2] = {nv > 0 && m[0] < g.M, nv > 0 && m[1] < g.M};
  float ws[8], cs[8], bs[8];
  if constexpr (PAIR) {
    if (threadIdx.x < 128) {
      const bool cols = threadIdx.x >= 64;   // (uniform over a wave)
      const int64_t at = (cols ? n0 : m0) + lane, end = cols ? g.N : g.M;
      scales[cols][lane] = (cols ? g.w_scale : g.pair_rows)[at < end ? at : end - 1];
    }
  } else {
    load8<float>(g.w_scale + n, nv, ws);
  }
  column_terms(g.ep, n, nv, cs, bs);
  Raw8<O> res[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (ok[i] && g.ep.residual != nullptr && g.splits == 1)
      res[i] = load_raw8<O>(static_cast<const O*>(g.ep.residual) + off[i], nv);
  // Bytes of the depth before a stage, and of the whole: the main one's, or the pair's.
  auto depth = [&](int st, int& k, int& len) __attribute__((always_inline)) {
    const bool pair = PAIR && st >= n1;   // (uniform)
    k = (pair ? st - n1 : st) * 128, len = (int)(pair ? g.K2 * 2 : g.K);
    return pair;
  };
  // (Every stage issues four loads, those past the depth of its last bytes again:
  // with a number that depends on the lane, a use would wait for them all.)
  u32x4 v[AHEAD][4];
  auto load = [&](int st, u32x4 (&to)[4]) __attribute__((always_inline)) {
    int k, len;
    const bool pair = depth(st < st1 ? st : st1 - 1, k, len);
    k += c * 16;
    const int at = k + 16 <= len ? k : len - 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = *reinterpret_cast<const u32x4_any*>((PAIR && pair ? p2[i] : p[i]) + at);
  };
  // (in the order of their uses, and so in the loop)
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) {
    load(st0 + j, v[j]);
    __builtin_amdgcn_sched_barrier(0);
  }
  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  // Values 4q to 4q + 3 of a lane are columns 8q + 4 fg and on of row fr. With a pair
  // the sums are scaled before its products are added, as in the other tiles.
  auto scaled = [&]() __attribute__((always_inline)) {
    const float rs = scales[0][wm * 32 + fr];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 w4 = *reinterpret_cast<const f32x4*>(&scales[1][wn * 32 + 8 * q + 4 * fg]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[4 * q + e] = (float)__float_as_int(acc[4 * q + e]) * rs * w4[e] * g.inv_s;
    }
  };
  auto stage = [&](int j, int st, auto more) __attribute__((always_inline)) {
    char* buf = lds + (j & 1) * BUF;
    int k, len;
    const bool pair = depth(st, k, len);
    if (k + 128 > len) {   // (uniform)
      const int over = k + c * 16 + 16 - len;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = dropped(v[j][i], over < 0 ? 0 : (over < 16 ? over : 16));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r + 32 * i;   // (b's rows behind a's)
      *reinterpret_cast<u32x4*>(buf + row * 128 + (c ^ ((row >> 1) & 7)) * 16) = v[j][i];
    }
    if constexpr (decltype(more)::value) load(st + AHEAD, v[j]);
    // (the waves a stage ahead write the other half, which all have read by now)
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    barrier_keep_loads();
    if (PAIR && pair && st == (n1 > st0 ? n1 : st0)) scaled();
    u32x4 fa[4], fb[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int at = ((s * 2 + fg) ^ ((fr >> 1) & 7)) * 16;
      fa[s] = *reinterpret_cast<const u32x4*>(buf + (wm * 32 + fr) * 128 + at);
      fb[s] = *reinterpret_cast<const u32x4*>(buf + (64 + wn * 32 + fr) * 128 + at);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {   // (turned: a lane holds a row's columns)
      if (PAIR && pair)
        acc = Op<TP>::run(&fb[s], &fa[s], acc);
      else
        acc = Op<int8x_t>::run(&fb[s], &fa[s], acc);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  int base = st0;
  for (; base + AHEAD <= st1; base += AHEAD) {
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) stage(j, base + j, Tag<true>{});
  }
#pragma unroll
  for (int j = 0; j + 1 < AHEAD; ++j)
    if (base + j < st1) stage(j, base + j, Tag<false>{});   // (uniform)
  __syncthreads();
  if constexpr (PAIR) {
    if (st1 <= n1) scaled();
    acc *= g.s;
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = (float)__float_as_int(acc[e]);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *reinterpret_cast<f32x4*>(lds + ((wm * 32 + fr) * LD + wn * 32 + 8 * q + 4 * fg) * 4) =
        f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  float f[16];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[8 * i + e] = reinterpret_cast<const float*>(lds)[(r + 32 * i) * LD + c * 8 + e];
      if constexpr (!PAIR) f[8 * i + e] *= ws[e];
    }
  if (g.splits > 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = f[8 * i + e];
      if (ok[i]) store8<float>(g.part + (int64_t)split * g.M * g.N + off[i], nv, o);
    }
  } else {
    epilogue_rows<O, 2>(g.ep, f, cs, bs, m, off, ok, nv, res);
  }
}

template <typename O>
hipError_t launch_any(GemmArgs g, hipStream_t st) {
  split_stages(g, 128, 64);
  g.n_mt = (int)((g.M + 63) / 64), g.n_nt = (int)((g.N + 63) / 64);
  const dim3 grid((unsigned)((int64_t)g.n_mt * g.n_nt * g.splits)), block(256);
  if constexpr (sizeof(O) == 2) {
    if (g.K2 > 0)
      hipLaunchKernelGGL((int8_any_kernel<O, true>), grid, block, 0, st, g);
    else
      hipLaunchKernelGGL((int8_any_kernel<O, false>), grid, block, 0, st, g);
  } else {
    hipLaunchKernelGGL((int8_any_kernel<O, false>), grid, block, 0, st, g);
  }
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || g.splits == 1 ? e : launch_join<O>(g, st);
}

template <typename O>
hipError_t launch(GemmArgs g, int cfg, hipStream_t st) {
  if (cfg == kAny64) return launch_any<O>(g, st);
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
