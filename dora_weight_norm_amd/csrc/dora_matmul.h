// The matrix product's arguments and plan (host side and kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dora {

// What follows the product, per element:
//   u = row_scale[m] * acc;  z = col_scale[n] * u + bias[n];  y = act(z) + residual
struct Epilogue {
  const float* row_scale;
  const float* col_scale;
  const float* bias;
  const void* residual;
  void* y;
  void* u;
  int act;
};

// One product acc[m][n] = sum_k a[m][k] b[n][k] + s sum_l a2[m][l] b2[n][l],
// operands with row strides in elements. A transposed operand is stored
// [k][row] instead (its stride is that of a k row).
struct GemmArgs {
  const void* a;
  const void* b;
  int64_t lda, ldb, K;
  const void* a2;
  const void* b2;
  int64_t lda2, ldb2, K2;
  float s;
  int64_t M, N;
  int n_mt, n_nt;          // tiles
  int splits;              // parts of the depth
  int stages;              // stages of the whole depth
  int stages_per_split;
  float* part;             // [splits][M][N] fp32 partial sums (splits > 1)
  Epilogue ep;
};

// Kernels: tiles of 256, 128 or 64 rows and columns, or the few-rows kernel on
// 8 rows by 16 columns, 16 by 16 or 32 by 32.
enum MatmulTile : int { kTile256 = 0, kTile128 = 1, kTile64 = 2, kFew8 = 3, kFew16 = 4, kFew32 = 5 };

struct MatmulPlan {
  int cfg;
  int splits;
  int64_t ldx, ldw, ldt, ldb;                  // row strides in elements of what the kernel reads
  bool pack_x, pack_w, pack_t, pack_b;         // copied into the workspace at that stride first
  size_t off_x, off_w, off_t, off_b, off_part;
  size_t ws_bytes;
};

// The product's plan; `al` is a bit mask of the operands whose pointers are
// 16-byte aligned (1 x, 2 w, 4 t, 8 b).
MatmulPlan plan_matmul(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int al);

struct MatmulBackwardPlan {
  bool du_direct;                               // du is written into the caller's array alone
  bool direct;                                  // the products read x, w and du in their own layout,
  bool copy;                                    // x and w from copies with a row stride of ldk
  int64_t rows;                                 // row blocks of the element-wise pass
  int64_t ldn, ldm, ldk;                        // padded N, M and K
  int cfg_dx, cfg_dw, splits_dx, splits_dw;
  size_t off_du, off_dut, off_wt, off_xt, off_sum, off_part;
  size_t ws_bytes;
};
MatmulBackwardPlan plan_matmul_backward(int64_t M, int64_t N, int64_t K, int dtype, bool need_dx, bool need_dw,
                                        bool need_sums, bool du_direct, bool aligned_xw);

hipError_t launch_matmul(const MatmulPlan& p, const void* x, const void* w, int dtype, int64_t M, int64_t N,
                         int64_t K, const void* t, const void* b, int64_t r, float s, const Epilogue& ep,
                         int out_dtype, char* ws, hipStream_t st);
hipError_t launch_matmul_backward(const MatmulBackwardPlan& p, const void* dy, const void* u, const void* x,
                                  const void* w, int dtype, int64_t M, int64_t N, int64_t K, const float* row_scale,
                                  const float* col_scale, const float* bias, int act, void* du, void* dx, void* dw,
                                  float* dbias, float* dcol, char* ws, hipStream_t st);

}  // namespace dora
