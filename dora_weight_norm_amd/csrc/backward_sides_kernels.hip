// What a product's backward needs between its element-wise pass and its products,
// in one launch: the sums over the rows, int8 rows brought back to 16 bits, and the
// transposed copies that fp32 products read. The parts do not depend on one
// another, and a launch costs 4 us of the host's time and as much on the GPU, which
// is what small products take. Measured with u, x and w as int8 rows, a launch for
// each against this: 64 x 128 x 256 fp32 40.8, 29.1 us (34.1, 17.5 on the GPU);
// 1024^3 fp32 87.7, 69.5; 1000 x 777 x 1500 bf16 50.4, 46.8; 4096^3 bf16 276.7,
// 275.4. Large copies run at the memory's rate.
#include "dora_matmul.h"
#include "int8_rows_device.h"

namespace dora {

namespace {

// The first `sums` workgroups add up columns; each of the others' four groups of
// 256 threads walks rows.
template <typename T, bool STREAM>
__global__ __launch_bounds__(kSumThreads) void rows_back_kernel(ColumnSum sum, unsigned sums, UnpackJob a, UnpackJob b,
                                                                RowSteps s, int64_t ld) {
  if (blockIdx.x < sums) return column_sum(sum, blockIdx.x);
  const unsigned group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  unpack_rows<T, STREAM, true>(a, b, s, ld, (blockIdx.x - sums) * 4 + group, (gridDim.x - sums) * 4, threadIdx.x & 255);
}

struct TurnJob {
  const float* src;     // or
  const uint8_t* q;     // int8 rows
  const float* scale;
  int64_t groups;
  int shift;
  int64_t rows, cols, lsrc, ld;
  float* dst;
  unsigned tiles;       // 64 x 64
};
struct TurnJobs {
  TurnJob job[3];
};

// (workgroups of the copies, each with as many tiles as it takes: a launch holds
// less than 2^32 threads)
constexpr unsigned kMostTurns = 1u << 16;

__global__ __launch_bounds__(kSumThreads) void turn_kernel(ColumnSum sum, unsigned sums, TurnJobs jobs, unsigned tiles) {
  __shared__ float tile[64][65];
  if (blockIdx.x < sums) return column_sum(sum, blockIdx.x);
  for (unsigned at = blockIdx.x - sums; at < tiles; at += gridDim.x - sums) {   // (uniform)
    unsigned blk = at;
    int i = 0;
    for (; i < 2 && blk >= jobs.job[i].tiles; ++i) blk -= jobs.job[i].tiles;
    const TurnJob& j = jobs.job[i];
    const unsigned nr = (unsigned)((j.ld + 63) / 64);   // (of the copy's stride, so that its padding is written)
    const int64_t r0 = (int64_t)(blk % nr) * 64, c0 = (int64_t)(blk / nr) * 64;
    const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
    constexpr int kStep = kSumThreads / 64;
#pragma unroll
    for (int k = 0; k < 64; k += kStep) {
      const int64_t r = r0 + k + ty, c = c0 + tx;
      float v = 0.f;
      if (r < j.rows && c < j.cols) {
        if (j.q)
          v = (float)(int8_t)j.q[r * j.lsrc + c] * j.scale[r * j.groups + (c >> j.shift)];
        else
          v = j.src[r * j.lsrc + c];
      }
      tile[k + ty][tx] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 64; k += kStep) {
      const int64_t c = c0 + k + ty, r = r0 + tx;
      if (c < j.cols && r < j.ld) j.dst[c * j.ld + r] = tile[tx][k + ty];
    }
    __syncthreads();
  }
}

template <typename T>
void rows_back(const ColumnSum& sum, unsigned sums, const BackwardSides& b, int64_t M, int64_t N, int64_t K, int64_t ldk,
               hipStream_t st) {
  const UnpackJob w = unpack_job(b.w8, b.w16 ? N : 0, K, b.w16, b.w_folded);
  const UnpackJob x = unpack_job(b.x8, b.x16 ? M : 0, K, b.x16, b.x_folded);
  const int64_t rows = w.T + x.T;
  const RowSteps s = row_steps(rows, K, 0, Elem<T>::epc, 1);
  const dim3 grid(sums + (row_groups(s) + 3) / 4), block(kSumThreads);
  if (rows * K * (int64_t)sizeof(T) > kStreamBytes && K % 128 == 0)
    hipLaunchKernelGGL((rows_back_kernel<T, true>), grid, block, 0, st, sum, sums, w, x, s, ldk);
  else
    hipLaunchKernelGGL((rows_back_kernel<T, false>), grid, block, 0, st, sum, sums, w, x, s, ldk);
}

}  // namespace

hipError_t launch_backward_sides(const BackwardSides& b, int64_t M, int64_t N, int64_t K, int64_t ldk, int dtype,
                                 hipStream_t st) {
  const bool back = K > 0 && ((b.w16 && N > 0) || (b.x16 && M > 0));
  const unsigned sums = b.want_sums ? sum_groups(2 * N) : 0;
  const ColumnSum sum{b.part, b.n_part, 2 * N, b.dbias, N, b.dcol};
  if (b.n_turned > 0) {
    TurnJobs jobs{};
    unsigned tiles = 0;
    for (int i = 0; i < b.n_turned; ++i) {
      const Turned& t = b.turned[i];
      const unsigned n = (unsigned)((t.ld + 63) / 64 * ((t.cols + 63) / 64));
      jobs.job[i] = TurnJob{static_cast<const float*>(t.src), t.rows8.q, t.rows8.scale, scales_of(t.cols, t.rows8.group),
                            group_shift(t.rows8.group), t.rows, t.cols, t.lsrc, t.ld, static_cast<float*>(t.dst), n};
      tiles += n;
    }
    const unsigned groups = tiles < kMostTurns ? tiles : kMostTurns;
    hipLaunchKernelGGL(turn_kernel, dim3(sums + groups), dim3(kSumThreads), 0, st, sum, sums, jobs, tiles);
  } else if (back) {
    if (dtype == 0)
      rows_back<bf16_t>(sum, sums, b, M, N, K, ldk, st);
    else
      rows_back<f16_t>(sum, sums, b, M, N, K, ldk, st);
  } else {
    return sums ? launch_column_sum(b.part, b.n_part, 2 * N, b.dbias, N, b.dcol, st) : hipSuccess;
  }
  return hipGetLastError();
}

}  // namespace dora
