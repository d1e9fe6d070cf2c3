// Matrix product with a fused epilogue on gfx950, and its backward.
//
//   u = row_scale[m] * (sum_k x[m,k] w[n,k] + s sum_l t[m,l] b[n,l])
//   y = act(col_scale[n] * u + bias[n]) + residual[m,n]
//
// bf16, fp16, fp32 or e4m3 operands on the matrix cores with fp32
// accumulation. The low-rank pair (t, b) runs through the same accumulators
// first, which are then multiplied by s, so that the adapter costs r more
// columns of depth and no pass over memory.
//
// Measured (MI355X, one box): 8192 x 8192 x 8192 with r = 384 in bf16 908 us,
// 1.27 PFLOP/s (the vendor's product alone, without r, 686 us); 8192 x 28672 x
// 8192 in e4m3 1.48 ms, 2.60 PFLOP/s (1.20 ms); 4096^3 with r = 64 113 us
// (87 us without); one token at 8192 x 8192 25 us, 5.6 TB/s (29 us); the
// backward at 4096^3 254 us, 1.08 PFLOP/s (the vendor's two products 219 us).
// On random operands the matrix cores sustain 1.73 PFLOP/s in bf16.
#include "dora_rows.h"
#include "matmul_device.h"

namespace dora {

namespace {

// Element-wise part of the backward: z from u, dz = dy act'(z), du = row_scale
// col_scale dz (rounded to the storage type: it is the operand of both
// products, which the matrix cores take in 16 bits), and this row block's sums
// of dz and dz u over its rows, in increasing order (u holds the row scale).
// U8: u is held as int8 rows (a strip of eight columns lies in one group).
struct SavedU {
  const uint8_t* q;
  const float* scale;
  int64_t groups;
  int shift;
};

// FOLD: beside du, or in its place, the operands of products whose other one is int8
// rows with one scale a row: du times the scales' significands (scale_parts.h), of w's rows
// for dx (du_n) and of x's for dw (du_m), rounded once, from which the rows' integers
// then take no rounding of their own. Either may be null, and du too.
template <typename T>
struct Folded {
  const float* n_scale;
  T* du_n;
  const float* m_scale;
  T* du_m;
};

template <typename T, bool U8, bool FOLD, bool KEEP>
__global__ __launch_bounds__(256) void matmul_bwd_kernel(const T* dy, const T* u, SavedU u8, const float* row_scale,
                                                         const float* col_scale, const float* bias, int act, int64_t M,
                                                         int64_t N, T* du, int64_t ldu, T* du2, Folded<T> fold,
                                                         float* sums) {
  __shared__ float lanes[16][256];
  const int64_t strip = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t n = strip * 8;
  const int ly = threadIdx.y, nl = blockDim.y;
  const int nv = (int)(N - n < 8 ? (N - n < 0 ? 0 : N - n) : 8);
  float cs[8], bs[8], sb[8], sc[8], fn[FOLD ? 8 : 1];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = (col_scale && e < nv) ? col_scale[n + e] : 1.f;
    bs[e] = (bias && e < nv) ? bias[n + e] : 0.f;
    sb[e] = sc[e] = 0.f;
    if constexpr (FOLD) fn[e] = fold.du_n && e < nv ? fold_factor<T>(fold.n_scale[n + e]) : 0.f;
  }
  // Four rows' loads are in flight at a time, and as int8 rows, which are fewer
  // bytes of u, the next four's too.
  constexpr int U = 4;
  struct Rows {
    Raw8<T> y[U], u[U8 ? 1 : U];
    uint32_t q[U8 ? U : 1][2];
    float s[U8 ? U : 1];
  };
  const int64_t step = (int64_t)gridDim.y * nl;
  auto load = [&](Rows& r, int64_t m0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t m = m0 + i * step;
      if (m < M) {
        // (what the products read next, du or with KEEP dy, is to stay in the caches)
        r.y[i] = load_raw8<T, !KEEP>(dy + m * N + n, nv);
        if constexpr (U8) {
          // (through the caches: 27.6 and 29.7 us at 4096 x 4096 with SiLU, sums included)
          load_row_bytes<8>(u8.q + m * N, n, N, r.q[i]);
          r.s[i] = u8.scale[m * u8.groups + (n >> u8.shift)];
        } else {
          r.u[i] = load_raw8<T, true>(u + m * N + n, nv);
        }
      }
    }
  };
  auto run = [&](const Rows& r, int64_t m0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t m = m0 + i * step;
      if (m >= M) continue;
      const float rs = row_scale ? row_scale[m] : 1.f;
      float y[8], v[8], o[8];
      unpack8<T>(r.y[i], y);
      if constexpr (U8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)(r.q[i][e / 4] >> (8 * (e % 4))) * r.s[i];
      } else {
        unpack8<T>(r.u[i], v);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(cs[e], v[e], bs[e]);
      slope_all<8, std::is_same<T, float>::value>(o, act);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dz = y[e] * o[e];
        sb[e] += dz;
        sc[e] = fmaf(dz, v[e], sc[e]);
        o[e] = cs[e] * dz * rs;
      }
      if (du2) store8<T>(du2 + m * N + n, nv, o);
      // (a padded row's tail, up to the next strip of eight, is written as zeros)
      auto put = [&](T* to, float (&v)[8]) __attribute__((always_inline)) {
        if (nv < 8 && ldu > N) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e >= nv) v[e] = 0.f;
          store8<T>(to + m * ldu + n, (int)(ldu - n < 8 ? ldu - n : 8), v);
        } else {
          store8<T>(to + m * ldu + n, nv, v);
        }
      };
      if constexpr (FOLD) {
        if (fold.du_n) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = o[e] * fn[e];
          put(fold.du_n, f);
        }
        if (fold.du_m) {
          const float fm = fold_factor<T>(fold.m_scale[m]);
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = o[e] * fm;
          put(fold.du_m, f);
        }
        if (du) put(du, o);
      } else {
        put(du, o);
      }
    }
  };
  const int64_t first = (int64_t)blockIdx.y * nl + ly;
  if constexpr (U8) {
    Rows a, b;
    if (nv > 0) load(a, first);
    for (int64_t m0 = first; nv > 0 && m0 < M; m0 += 2 * U * step) {
      load(b, m0 + U * step);
      run(a, m0);
      load(a, m0 + 2 * U * step);
      run(b, m0 + U * step);
    }
  } else {
    for (int64_t m0 = first; nv > 0 && m0 < M; m0 += U * step) {
      Rows r;
      load(r, m0);
      run(r, m0);
    }
  }
  if (sums == nullptr) return;   // uniform
  const int at = ly * blockDim.x + threadIdx.x;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lanes[e][at] = sb[e];
    lanes[8 + e][at] = sc[e];
  }
  __syncthreads();
  if (ly != 0 || nv <= 0) return;
  for (int k = 1; k < nl; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sb[e] += lanes[e][k * blockDim.x + threadIdx.x];
      sc[e] += lanes[8 + e][k * blockDim.x + threadIdx.x];
    }
  // partial row: [dbias | dcol_scale] of this row block
  float* p = sums + (int64_t)blockIdx.y * 2 * N;
  store8<float>(p + n, nv, sb);
  store8<float>(p + N + n, nv, sc);
}

constexpr int kCUs = 256;

constexpr int kRowBlocks = 512;   // workgroups of the element-wise backward

int tile_rows(int cfg) { return cfg == kTile256 ? 256 : (cfg == kTile128 ? 128 : 64); }
// Elements of a stage's 128 bytes of depth.
int stage_depth(int dtype) { return dtype == 1 ? 32 : (dtype >= 3 ? 128 : 64); }
int elem_size(int dtype) { return dtype == 1 ? 4 : (dtype >= 3 ? 1 : 2); }
// Elements of the low-rank pair.
int pair_size(int dtype) { return dtype == kInt8Operands ? 2 : elem_size(dtype); }
int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Workgroups of 16 x 16 of the few-rows kernel.
int64_t few_blocks(int64_t M, int64_t N) { return up(M, 16) / 16 * (up(N, 16) / 16); }
// The most parts of the depth that n workgroups of it are split into: while
// they do not fill the chip and each wave keeps four steps.
int64_t few_splits(int64_t n, int64_t stages) {
  int64_t s = n >= kCUs || n < 1 ? 1 : kCUs / n;
  if (s > stages / 16) s = stages / 16;
  return s < 1 ? 1 : s;
}
// 17 to 32 rows take 32 x 32, which reads w once instead of twice, where 16 x
// 16 would need a second round (48 x 4096 x 4096, two rounds and more: 27 us
// against 22; 32 x 1001 x 1024 bf16: 5.1 us in 16 x 16, 8.6 in 32 x 32). So do
// long depths of more than 512 columns, from 64 stages on for rows off the
// 16-byte grid, whose every load takes two lines, and 128 for others, if a
// workgroup of 16 x 16 would have 48 of them or more. Measured, 16 x 16 against
// 32 x 32, us on the GPU:
//   17 and 32 x 1001 x 8189 fp16   25.2, 20.3 and 24.5, 23.6
//   17 and 32 x 2048 x 4093 fp16   23.9, 19.0 and 23.5, 21.8
//   17 and 32 x 1500 x 3581 fp16   21.9, 21.9 and 22.1, 25.3 (56 stages)
//   17 and 32 x 1001 x 8192 bf16   15.6, 14.0 and 15.6, 15.2
//   17 and 32 x 2048 x 8192 bf16   19.9, 17.5 and 18.6, 19.3
//   17 and 32 x 2048 x 4096 bf16   11.0, 11.0 and 10.8, 12.7 (64 stages)
//   17 and 32 x 2048 x 16384 e4m3  19.1, 15.2 and 18.0, 17.9
//   17 and 32 x 256 x 32765 fp16   26.4, 28.0 and 25.9, 31.5
// fp32, whose matrix instructions are the slow part, gains nowhere (17 x 2048
// x 4096: 20.4, 22.1).
bool few_wide(int64_t M, int64_t N, int64_t stages, int dtype, bool on_grid) {
  if (M <= 16 || M > 32) return false;
  const int64_t n = few_blocks(M, N);
  if (n > kCUs) return true;
  return dtype != 1 && n > 64 && stages >= (on_grid ? 128 : 64) && stages >= 48 * few_splits(n, stages);
}

// `few`: the most stages that a workgroup of the few-rows kernel may take where
// there are more than 32 rows, 0 where it cannot run. Rows off the 16-byte
// grid are copied for the tiles and not here, where their loads cost more from
// about 24 stages on (128 x 256 x 4093 fp16, 32 a workgroup: 17.2 us, 15.9 as
// a tile).
constexpr int kFewOnGrid = 64, kFewOffGrid = 24;
void choose_tile(int64_t M, int64_t N, int64_t stages, int dtype, int few, int* cfg, int* splits) {
  if (few > 0 && (M <= 32 || (stages >= 4 && few_blocks(M, N) <= kCUs))) {
    // Up to 32 rows come here at any depth and alignment (17 x 1001 x 8189
    // fp16: 20 us, 32 as a tile behind copies; 32 x 8192 x 4093: 45.5, 40.9).
    // More than 32 rows come here while one round of workgroups covers the
    // result and none has more than `few` stages
    // (64-row tile against this, us on the GPU: 64 x 256 x 256 fp32 9.6, 5.6;
    // 256 x 256 x 1024 bf16 7.1, 4.8; 64 x 1001 x 4096 bf16 16.7, 12.4; but
    // 64 x 4096 x 1024 bf16, four rounds, 7.2, 11.6). Below four stages the
    // two differ by 1 us or less, which the host's share of the call hides.
    const bool wide = few_wide(M, N, stages, dtype, few == kFewOnGrid);
    const int64_t s = few_splits(wide ? up(N, 32) / 32 : few_blocks(M, N), stages);
    if (M <= 32 || stages <= few * s) {
      *cfg = M <= 8 ? kFew8 : (wide ? kFew32 : kFew16);
      *splits = (int)s;
      return;
    }
  }
  // The tile and the split that a model of the time puts first, in cycles. A
  // compute unit holds one workgroup of a 256-row tile or two of the others; a
  // stage of each costs it t^2 / 32 of matrix instructions (fp32: 16 times
  // that) or 4 t of loads, and a workgroup waits about kStageWait for a stage
  // from memory with a ring of two stages ahead (measured: 1500 to 1900 cycles
  // a stage where 256 workgroups of either small tile run), half of that with
  // four. The parts of a split are added by a second launch that reads them
  // all.
  constexpr double kStageWait = 1600, kJoinFixed = 12000, kBytesPerCycle = 2000;
  double best = 0;
  *cfg = kTile64, *splits = 1;
  for (int c = kTile256; c <= kTile64; ++c) {
    if (c == kTile256 && dtype == 1) continue;   // (fp32 has no such kernel: its matrix instructions are slow)
    const int t = tile_rows(c), fit = c == kTile256 ? 1 : 2;
    const int64_t n = up(M, t) / t * (up(N, t) / t);
    const double work = (dtype == 1 ? 16.0 : 1.0) * t * t / 32, load = 4.0 * t, busy = work > load ? work : load;
    const double wait = c == kTile64 ? kStageWait / 2 : kStageWait;
    for (int s = 1; s <= 32 && (s == 1 || s <= stages / 4); ++s) {
      const int64_t groups = n * s, rounds = (groups + kCUs * fit - 1) / (kCUs * fit);
      const int64_t last = groups - (rounds - 1) * kCUs * fit;   // workgroups of the last round
      auto round = [&](int64_t g) {
        const double here = (double)((g + kCUs - 1) / kCUs) * busy;
        return (double)((stages + s - 1) / s) * (here > wait ? here : wait) + 4000 + 16 * t;
      };
      double time = (double)(rounds - 1) * round((int64_t)kCUs * fit) + round(last);
      if (s > 1) time += kJoinFixed + 8.0 * s * (double)M * (double)N / kBytesPerCycle;
      if (best == 0 || time < best) best = time, *cfg = c, *splits = s;
    }
  }
}

// Whether a product of 8-bit integers with few rows goes to the tiles all the
// same. They bring rows into shared memory in whole lines without a register,
// which 32 rows of w in pieces of 16 bytes do not reach, and have more of w on
// its way than blocks of 16 columns do, at shallow depths or where the walking
// kernel ends; rows whose length is off the 16-byte grid stay. (A w at an address
// off it: int8_in_place.)
// Measured, the few-rows or walking kernel against the tiles, us on the GPU:
//   17 and 32 x 28672 x 8192   76.6, 44.3 and 87.3, 46.2
//   17 and 32 x  8192 x 8192   21.9, 19.0 and 24.5, 19.3
//   17 and 32 x  8192 x 1024    8.6,  6.1 and  9.6,  6.2
//   17 and 32 x  4096 x 4096   12.4, 12.7 and 13.8, 13.8
//   17 and 32 x  2048 x 16384  18.5, 17.2 and 20.4, 17.8
//   17 and 32 x  4096 x 32768  36.3, 48.2 and 41.0, 47.9 (rows 32 KB apart)
//    1 and 16 x 28672 x 1024   13.1,  9.8 and 14.1,  9.9
//    1 and 16 x 28672 x 2048   16.4, 14.8 and 16.8, 14.9
//    1 and 16 x 28672 x 4096   23.1, 26.2 and 26.0, 26.3
//    1 and 16 x 16384 x 2048   10.4,  9.7 and 11.3,  9.8
//    1 and 16 x 12288 x 2048    8.7,  9.1 and  9.3,  9.2
//    1 and 16 x  8192 x 512     4.8,  5.3 and  5.3,  5.3
//    9 and 16 x  8192 x 16384  29.1, 35.7 and 33.5, 36.1 (8 rows for 9)
//    9 and 16 x  8192 x 24576  41.2, 41.4 and 48.4, 41.9
//    9 and 16 x 12288 x 12288  32.7, 37.5 and 37.8, 37.8
//    9 and 16 x 28672 x 12288  69.1, 72.0 and 81.9, 74.4
bool int8_tiles(int64_t M, int64_t N, int64_t K) {
  if (M > 32 || K == 0 || K % 16 != 0) return false;
  if (M > 16) return few_wide(M, N, up(K, 128) / 128, kInt8Operands, true);
  return (N >= 4 * 16 * kCUs && K <= 2048) || (M > 12 && K > 8192 && N * K > (int64_t)1 << 27);
}

// Whether 64-row tiles of 8-bit integers take rows off the 16-byte grid as they are
// (int8_any_kernel), or behind copies: a copy costs a launch and its bytes, loads
// through registers half as much again for each stage of each tile. A pair's
// copies are small. (By sizes alone: a workspace for operands at any address serves
// them at all.) Measured, behind copies against as they are, us of the whole call:
//    333 x 1001 x  777, r = 24   16.5, 10.9      2304 stages of all tiles
//     64 x 8192 x 8189           44.2, 22.2      8192
//    128 x 8192 x 8189           48.2, 35.3     16384
//    256 x 4096 x 8191           36.1, 35.1     16384
//    500 x 4000 x 5001           39.9, 39.3     20160
//   1000 x 1700 x 8190           40.6, 49.1     27648
// the pair alone, by the stages of a workgroup,
//    128 x 8192 x  512, r = 390  14.9, 11.0     11
//   1000 x 1000 x 2000, r = 13   15.4, 13.7     17
//     64 x 8192 x 8192, r = 13   22.9, 19.9     17
//   1000 x 1000 x 4000, r = 13   18.7, 21.6     33
bool int8_anywhere(int64_t M, int64_t N, int64_t K, int64_t r, int splits) {
  if (K < 16 || (r > 0 && r < 8)) return false;
  const int64_t tiles = up(M, 64) / 64 * (up(N, 64) / 64), stages = up(K, 128) / 128 + up(r, 64) / 64;
  return tiles * stages <= 20000 && (K % 16 != 0 || stages <= 20 * splits);
}

// Whether a product whose result is one row of 64-row tiles takes a w off the
// 16-byte grid as it is: a copy writes and reads again what is read once here, in a
// workspace as large as w. Measured, behind copies against as they are, us of the
// whole call (w one byte off the grid, or rows of an odd length):
//   17 and 32 x  28672 x 8192   127, 93 and 129, 93 (few-rows kernel 200, 244)
//   17 and 32 x  28672 x 4096    60, 47 and  60, 48 (few-rows kernel 109, 132)
//   14        x  28672 x 8320   132, 91             (few-rows kernel 191)
//   33 and 64 x  28672 x 8189   132, 70 and 139, 81
//   32 and 64 x  8192 x 28672   135, 86 and 142, 89
//   64        x 100000 x 2000   144, 84
//  128        x  28672 x 8192   153, 169 and x 2000 38, 35 (two rows of tiles)
bool int8_in_place(int64_t M, int64_t K, int al) { return M <= 64 && K >= 16 && (K % 16 != 0 || !(al & 2)); }

// Whether the walking kernel takes a product of 8-bit integers: whole steps of
// 128 bytes, eight a wave at most, a pair of one step a wave in whole chunks, and
// two blocks of columns or more for a compute unit; up to 8 rows, for which the
// few-rows kernel reads fewer tokens, three, and depths of 2048 and more, since
// a block's bytes are all that a unit has on their way. Measured, the few-rows
// kernel against this, us on the GPU:
//    1, 8 and 16 x  8192 x 8192   13.1, 14.7; 15.2, 15.3; 19.5, 16.3
//    1, 8 and 16 x 12288 x 8192   21.6, 19.6; 22.3, 20.2; 27.7, 20.9
//    1, 8 and 16 x 28672 x 8192   43.0, 37.6; 48.1, 39.5; 59.0, 40.2
//    1, 8 and 16 x 16384 x 1024    7.8,  8.3;  8.7,  8.4; 10.4,  9.0
bool int8_walks(int64_t M, int64_t N, int64_t K, int64_t r) {
  if (M > 16 || K == 0 || K % 128 != 0 || K > 8192 || r > 512 || r % 8 != 0) return false;
  return M > 8 ? N >= 2 * 16 * kCUs : N >= 3 * 16 * kCUs && K >= 2048;
}

// The backward's products on operands as they lie (16-bit types): `b` stored
// [k][row], and with AT `a` too.
template <typename T, bool AT>
hipError_t launch_gemm_tr(GemmArgs g, int cfg, hipStream_t st) {
  split_stages(g, 64, 64);
  hipError_t e = hipErrorInvalidValue;
  if (cfg == kTile256) e = launch_tile<T, T, 2, 4, 4, 2, 2, false, AT, true>(g, st);
  if (cfg == kTile128) e = launch_tile<T, T, 2, 2, 2, 2, 2, false, AT, true>(g, st);
  if (cfg == kTile64) e = launch_tile<T, T, 2, 2, 1, 1, 4, false, AT, true>(g, st);
  return e != hipSuccess || g.splits == 1 ? e : launch_join<T>(g, st);
}

template <typename T, typename O>
hipError_t launch_gemm(GemmArgs g, int cfg, hipStream_t st) {
  if (cfg == kFew8) return launch_few_rows<T, O, 2, 1>(g, st);
  if (cfg == kFew16) return launch_few_rows<T, O, 2, 2>(g, st);
  if (cfg == kFew32) return launch_few_rows<T, O, 4, 4>(g, st);
  split_stages(g, 128 / Op<T>::esz, 128 / Op<T>::esz);
  hipError_t e = hipErrorInvalidValue;
  if (g.K2 > 0) {
    if constexpr (Op<T>::esz > 1) {   // (no pair in e4m3)
      if constexpr (Op<T>::esz == 2) {
        if (cfg == kTile256) e = launch_tile<T, O, 2, 4, 4, 2, 2, true>(g, st);
      }
      if (cfg == kTile128) e = launch_tile<T, O, 2, 2, 2, 2, 2, true>(g, st);
      if (cfg == kTile64) e = launch_tile<T, O, 2, 2, 1, 1, 4, true>(g, st);
    }
  } else {
    if constexpr (Op<T>::esz == 2) {
      if (cfg == kTile256) e = launch_tile<T, O, 2, 4, 4, 2, 2, false>(g, st);
    }
    if constexpr (Op<T>::esz == 1) {
      if (cfg == kTile256) e = launch_tile<T, O, 2, 2, 4, 4, 2, false>(g, st);
    }
    if (cfg == kTile128) e = launch_tile<T, O, 2, 2, 2, 2, 2, false>(g, st);
    if (cfg == kTile64) e = launch_tile<T, O, 2, 2, 1, 1, 4, false>(g, st);
  }
  return e != hipSuccess || g.splits == 1 ? e : launch_join<O>(g, st);
}

hipError_t gemm(const GemmArgs& g, int dtype, int out_dtype, int cfg, hipStream_t st) {
  switch (dtype) {
    case 0: return launch_gemm<bf16_t, bf16_t>(g, cfg, st);
    case 2: return launch_gemm<f16_t, f16_t>(g, cfg, st);
    case 1: return launch_gemm<float, float>(g, cfg, st);
    default:
      switch (out_dtype) {
        case 0: return launch_gemm<e4m3_t, bf16_t>(g, cfg, st);
        case 2: return launch_gemm<e4m3_t, f16_t>(g, cfg, st);
        default: return launch_gemm<e4m3_t, float>(g, cfg, st);
      }
  }
}

}  // namespace

MatmulPlan plan_matmul(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int al) {
  MatmulPlan p{};
  const int esz = elem_size(dtype), epc = 16 / esz, KT = stage_depth(dtype);
  size_t off = 0;
  const bool i8 = dtype == kInt8Operands, tiles = i8 && int8_tiles(M, N, K);
  choose_tile(M, N, up(K, KT) / KT, dtype, tiles ? 0 : (K % epc == 0 ? kFewOnGrid : kFewOffGrid), &p.cfg, &p.splits);
  const bool off_grid = K % 16 != 0 || (al & 3) != 3 || (r > 0 && (r % 8 != 0 || (al & 12) != 12));
  if (i8 && p.cfg == kTile64 && off_grid && int8_anywhere(M, N, K, r, p.splits)) p.cfg = kAny64;
  size_t least = 0;
  if (i8 && p.cfg < kFew8 && int8_in_place(M, K, al)) {
    p.cfg = kAny64;
    if (K % 16 == 0) least = plan_matmul(M, N, K, r, dtype, al | 2).ws_bytes;   // (a workspace for any address serves all)
  }
  if (i8 && !tiles && int8_walks(M, N, K, r)) p.cfg = M <= 8 ? kWalk8 : kWalk16, p.splits = 1;
  auto operand = [&](int64_t rows, int64_t depth, int es, int bit, bool* pack, int64_t* ld, size_t* at) {
    // (The few-rows kernel reads rows at any element address; the 64-row tile that
    // does takes none shorter than 16 bytes, which a pair's may be.)
    *pack = depth > 0 && (p.cfg < kFew8 ? depth % (16 / es) != 0 || !(al & bit) : p.cfg == kAny64 && depth < 16 / es);
    *ld = *pack ? up(depth, 16 / es) : depth;
    *at = off;
    if (*pack) off = up256(off + (size_t)(rows * *ld) * es);
  };
  const int es2 = pair_size(dtype);
  operand(M, K, esz, 1, &p.pack_x, &p.ldx, &p.off_x);
  operand(N, K, esz, 2, &p.pack_w, &p.ldw, &p.off_w);
  operand(M, r, es2, 4, &p.pack_t, &p.ldt, &p.off_t);
  operand(N, r, es2, 8, &p.pack_b, &p.ldb, &p.off_b);
  p.off_part = off;
  if (p.splits > 1) off = up256(off + (size_t)(p.splits * M * N) * 4);
  p.ws_bytes = off > least ? off : least;
  return p;
}

hipError_t launch_matmul(const MatmulPlan& p, const void* x, const void* w, int dtype, int64_t M, int64_t N,
                         int64_t K, const void* t, const void* b, int64_t r, float s, const Epilogue& ep,
                         const float* w_scale, int out_dtype, char* ws, hipStream_t st) {
  const int esz = elem_size(dtype), es2 = pair_size(dtype);
  PackJobs jobs{};
  if (p.pack_x) add_pack(jobs, &x, M, K * esz, p.ldx * esz, ws + p.off_x);
  if (p.pack_w) add_pack(jobs, &w, N, K * esz, p.ldw * esz, ws + p.off_w);
  if (p.pack_t) add_pack(jobs, &t, M, r * es2, p.ldt * es2, ws + p.off_t);
  if (p.pack_b) add_pack(jobs, &b, N, r * es2, p.ldb * es2, ws + p.off_b);
  const hipError_t e = launch_pack(jobs, st);
  if (e != hipSuccess) return e;
  GemmArgs g{};
  g.a = x, g.b = w, g.lda = p.ldx, g.ldb = p.ldw, g.K = K;
  g.a2 = r > 0 ? t : nullptr, g.b2 = r > 0 ? b : nullptr, g.lda2 = p.ldt, g.ldb2 = p.ldb;
  g.K2 = p.cfg == kAny64 && p.pack_t ? p.ldt : r;   // (with the zeros behind copies of such rows)
  g.s = s, g.M = M, g.N = N, g.splits = p.splits;
  g.part = reinterpret_cast<float*>(ws + p.off_part);
  g.ep = ep;
  if (dtype == kInt8Operands) {
    g.w_scale = w_scale;
    if (r > 0 || p.cfg == kWalk8 || p.cfg == kWalk16) {   // (the pair's products are added to scaled sums, and s multiplies both)
      g.pair_rows = ep.row_scale, g.ep.row_scale = nullptr;
      g.inv_s = 1.f / s;
    }
    return gemm_int8(g, out_dtype, p.cfg, st);
  }
  return gemm(g, dtype, out_dtype, p.cfg, st);
}

// Whether a product of so many rows reads int8 rows [depth][K] as they are held,
// or from 16-bit copies: the conversion makes its loop a tenth slower, the copies
// cost a launch and three bytes an element of the rows whatever the product, which
// is as much at 4096 rows. Measured, as held against copied, us of the whole call
// without sums, dw of M x N x K (N rows) and dx (M rows):
//    8192 x  384 x  8192    89, 116;   80,  90
//    8192 x  768 x  8192   133, 153;  122, 125
//    8192 x  384 x 28672   207, 315;  260, 302
//    2048 x 2048 x  2048    41,  44;   42,  44
//    4096 x 4096 x  4096   142, 142;  137, 139
//    8192 x 4096 x  8192   494, 489;  486, 479
//    8192 x 8192 x  8192   976, 927;  942, 899
static bool reads_rows8(int64_t rows, int64_t depth, int64_t K) {
  return rows <= 4096 || (double)(rows - 4096) * (double)depth * (double)K < 2.7e10;
}

MatmulBackwardPlan plan_matmul_backward(int64_t M, int64_t N, int64_t K, int dtype, bool need_dx, bool need_dw,
                                        bool need_sums, bool du_direct, bool aligned_xw, HeldForm x8, HeldForm w8) {
  MatmulBackwardPlan p{};
  p.x8 = x8 != kNotHeld && need_dw, p.w8 = w8 != kNotHeld && need_dx;
  p.fold_x = x8 == kHeldRows && need_dw && dtype != 1 && K > 0;
  p.fold_w = w8 == kHeldRows && need_dx && dtype != 1 && K > 0;
  // (where both products have operands of their own, du is the caller's alone)
  p.plain = !(p.fold_x || p.fold_w) || (need_dx && !p.fold_w) || (need_dw && !p.fold_x);
  const int esz = elem_size(dtype), epc = 16 / esz, KT = stage_depth(dtype);
  p.ldn = up(N, epc), p.ldm = up(M, epc);
  const int64_t strips = (N + 7) / 8, bx = (strips + 255) / 256;
  p.rows = bx > 0 ? kRowBlocks / bx : 1;
  if (p.rows < 1) p.rows = 1;
  if (p.rows > (M + 7) / 8) p.rows = (M + 7) / 8;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  p.du_direct = du_direct && N % epc == 0;
  p.off_du = take(p.du_direct || !p.plain ? 0 : (size_t)(M * p.ldn) * esz);
  p.off_dun = take(p.fold_w ? (size_t)(M * p.ldn) * esz : 0);
  p.off_dum = take(p.fold_x ? (size_t)(M * p.ldn) * esz : 0);
  p.off_sum = take(need_sums ? (size_t)(p.rows * 2 * N) * 4 : 0);
  // 16-bit products read du, w and x as they lie, copied to whole chunks where
  // their rows are none; fp32 ones (whose elements no transposing read takes)
  // read transposed copies.
  p.direct = dtype != 1;
  p.ldk = up(K, epc);
  p.copy = p.direct && (!aligned_xw || K % epc != 0);
  if (need_dx) choose_tile(M, K, up(N, KT) / KT, dtype, p.direct ? 0 : kFewOnGrid, &p.cfg_dx, &p.splits_dx);
  if (need_dw) choose_tile(N, K, up(M, KT) / KT, dtype, p.direct ? 0 : kFewOnGrid, &p.cfg_dw, &p.splits_dw);
  const bool chunks = p.direct && aligned_xw && K % 16 == 0;
  p.w8_tile = p.w8 && chunks && p.cfg_dx != kTile64 && reads_rows8(M, N, K);
  p.x8_tile = p.x8 && chunks && p.cfg_dw != kTile64 && reads_rows8(N, M, K);
  // (int8 rows are brought back at the copies' stride, as whole chunks, whether or not others are copied)
  const size_t w_bytes = (size_t)(N * p.ldk) * esz, x_bytes = (size_t)(M * p.ldk) * esz;
  const bool w_copy = p.w8 ? !p.w8_tile : p.copy, x_copy = p.x8 ? !p.x8_tile : p.copy;
  p.off_wt = take(!need_dx ? 0 : (p.direct ? (w_copy ? w_bytes : 0) : (size_t)(K * p.ldn) * esz));
  p.off_dut = take(need_dw && !p.direct ? (size_t)(N * p.ldm) * esz : 0);
  p.off_xt = take(!need_dw ? 0 : (p.direct ? (x_copy ? x_bytes : 0) : (size_t)(K * p.ldm) * esz));
  size_t part = 0;
  if (need_dx) {
    if (p.splits_dx > 1) part = (size_t)(p.splits_dx * M * K) * 4;
  }
  if (need_dw) {
    const size_t q = p.splits_dw > 1 ? (size_t)(p.splits_dw * N * K) * 4 : 0;
    part = q > part ? q : part;
  }
  p.off_part = take(part);
  p.ws_bytes = off;
  return p;
}

hipError_t launch_matmul_backward(const MatmulBackwardPlan& p, const void* dy, const void* u, const void* x,
                                  const void* w, int dtype, int64_t M, int64_t N, int64_t K, const float* row_scale,
                                  const float* col_scale, const float* bias, int act, void* du, void* dx, void* dw,
                                  float* dbias, float* dcol, const HeldInt8& held, char* ws, hipStream_t st) {
  const int esz = elem_size(dtype);
  hipError_t e = hipSuccess;
  // The element-wise pass writes du into the caller's array where that can be
  // the products' operand, else at a padded row stride into the workspace
  // (and into the caller's array beside it).
  char* d = !p.plain ? nullptr : (p.du_direct ? static_cast<char*>(du) : ws + p.off_du);
  void* du2 = p.plain && p.du_direct ? nullptr : du;
  // (without rows the workspace may be null: whether sums are wanted is not read off their address)
  const bool want_sums = dbias || dcol;
  float* sums = want_sums ? reinterpret_cast<float*>(ws + p.off_sum) : nullptr;
  // Without an activation or a row scale du is dy times a column's scale, which is a
  // row's of dw: dy itself is dw's operand then, and the scale multiplies the sums, so
  // that the rounding of x's values is the only one of an operand. (Where dy has the
  // layout, and is not du's place.)
  const bool of_dy = p.direct && p.x8 && !p.fold_x && act == 0 && row_scale == nullptr && col_scale != nullptr && dy != du &&
                     p.ldn == N && reinterpret_cast<uintptr_t>(dy) % 16 == 0;
  if (M > 0 && N > 0) {
    const int64_t strips = (N + 7) / 8;
    int64_t tx = up(strips, 64);
    if (tx > 256) tx = 256;
    const dim3 block((unsigned)tx, (unsigned)(256 / tx));
    const dim3 grid((unsigned)((strips + tx - 1) / tx), (unsigned)p.rows);
    const SavedU u8{held.u.q, held.u.scale, scales_of(N, held.u.group), group_shift(held.u.group)};
#define DORA_BWD_F(T, U8, FOLD, KEEP)                                                                                \
  hipLaunchKernelGGL((matmul_bwd_kernel<T, U8, FOLD, KEEP>), grid, block, 0, st, static_cast<const T*>(dy),                \
                     static_cast<const T*>(u), u8, row_scale, col_scale, bias, act, M, N, reinterpret_cast<T*>(d),   \
                     p.ldn, static_cast<T*>(du2),                                                                    \
                     (Folded<T>{held.w.scale, p.fold_w ? reinterpret_cast<T*>(ws + p.off_dun) : nullptr,             \
                                held.x.scale, p.fold_x ? reinterpret_cast<T*>(ws + p.off_dum) : nullptr}),           \
                     sums)
#define DORA_BWD_U(T, FOLD, KEEP)    \
  if (u8.q != nullptr)               \
    DORA_BWD_F(T, true, FOLD, KEEP); \
  else                               \
    DORA_BWD_F(T, false, FOLD, KEEP)
#define DORA_BWD(T)                  \
  if (p.fold_w || p.fold_x) {        \
    DORA_BWD_U(T, true, false);      \
  } else if (of_dy) {                \
    DORA_BWD_U(T, false, true);      \
  } else {                           \
    DORA_BWD_U(T, false, false);     \
  }
    switch (dtype) {
      case 0: DORA_BWD(bf16_t) break;
      case 2: DORA_BWD(f16_t) break;
      default: DORA_BWD_U(float, false, false); break;
    }
#undef DORA_BWD
#undef DORA_BWD_U
#undef DORA_BWD_F
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // The sums, and operands of the products that are not read as they lie: int8
  // rows in the storage type, transposed copies.
  BackwardSides side{};
  side.want_sums = want_sums && N > 0;
  side.part = sums, side.n_part = M > 0 ? (int)p.rows : 0, side.dbias = dbias, side.dcol = dcol;
  const bool w_back = p.direct && p.w8 && !p.w8_tile, x_back = p.direct && p.x8 && !p.x8_tile;
  if (w_back) side.w8 = held.w, w = side.w16 = ws + p.off_wt, side.w_folded = p.fold_w;
  if (x_back) side.x8 = held.x, x = side.x16 = ws + p.off_xt, side.x_folded = p.fold_x;
  if (!p.direct && M > 0 && K > 0 && N > 0) {
    if (dx) side.turn(w, held.w, N, K, K, p.ldn, ws + p.off_wt);
    if (dw) side.turn(d, Int8Rows{}, M, N, p.ldn, p.ldm, ws + p.off_dut);
    if (dw) side.turn(x, held.x, M, K, K, p.ldm, ws + p.off_xt);
  }
  e = launch_backward_sides(side, M, N, K, p.ldk, dtype, st);
  if (e != hipSuccess) return e;
  GemmArgs g{};
  g.part = reinterpret_cast<float*>(ws + p.off_part);
  if (p.direct) {
    if (p.copy) {
      PackJobs jobs{};
      if (dx && !p.w8) add_pack(jobs, &w, N, K * esz, p.ldk * esz, ws + p.off_wt);
      if (dw && !p.x8) add_pack(jobs, &x, M, K * esz, p.ldk * esz, ws + p.off_xt);
      e = launch_pack(jobs, st);
      if (e != hipSuccess) return e;
    }
    const int64_t ldu = p.du_direct ? N : p.ldn;
    const int64_t ldw = p.copy || p.w8 ? p.ldk : K, ldx = p.copy || p.x8 ? p.ldk : K;
    auto rows8 = [&](const Int8Rows& r, bool folded, bool across, int cfg) {
      g.b = r.q, g.ldb = K, g.b_scale = r.scale, g.b_groups = scales_of(K, r.group), g.b_shift = group_shift(r.group);
      g.b_folded = folded;
      return gemm_rows8(g, dtype, across, cfg, st);
    };
    // dx: du along the depth, w across it; dw: both across it.
    if (dx && M > 0 && K > 0) {
      g.a = p.fold_w ? ws + p.off_dun : d, g.lda = p.fold_w ? p.ldn : ldu;
      g.b = w, g.ldb = ldw, g.K = N, g.M = M, g.N = K, g.splits = p.splits_dx;
      g.ep.y = dx;
      if (p.w8_tile)
        e = rows8(held.w, p.fold_w, false, p.cfg_dx);
      else
        e = dtype == 0 ? launch_gemm_tr<bf16_t, false>(g, p.cfg_dx, st) : launch_gemm_tr<f16_t, false>(g, p.cfg_dx, st);
      if (e != hipSuccess) return e;
    }
    if (dw && N > 0 && K > 0) {
      g.a = p.fold_x ? ws + p.off_dum : d, g.lda = p.fold_x ? p.ldn : ldu;
      if (of_dy) g.a = dy, g.lda = N, g.ep.row_scale = col_scale;
      g.b = x, g.ldb = ldx, g.K = M, g.M = N, g.N = K, g.splits = p.splits_dw;
      g.ep.y = dw;
      if (p.x8_tile)
        e = rows8(held.x, p.fold_x, true, p.cfg_dw);
      else
        e = dtype == 0 ? launch_gemm_tr<bf16_t, true>(g, p.cfg_dw, st) : launch_gemm_tr<f16_t, true>(g, p.cfg_dw, st);
    }
    return e;
  }
  if (dx && M > 0 && K > 0) {
    g.a = d, g.b = ws + p.off_wt, g.lda = p.ldn, g.ldb = p.ldn, g.K = N, g.M = M, g.N = K, g.splits = p.splits_dx;
    g.ep.y = dx;
    e = gemm(g, dtype, dtype, p.cfg_dx, st);
    if (e != hipSuccess) return e;
  }
  if (dw && N > 0 && K > 0) {
    g.a = ws + p.off_dut, g.b = ws + p.off_xt, g.lda = p.ldm, g.ldb = p.ldm, g.K = M, g.M = N, g.N = K;
    g.splits = p.splits_dw;
    g.ep.y = dw;
    e = gemm(g, dtype, dtype, p.cfg_dw, st);
  }
  return e;
}

}  // namespace dora
