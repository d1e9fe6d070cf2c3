// The matrix product's arguments and plan (host side and kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dora_launch.h"

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
  // 8-bit integers: the columns' scales; with a pair, and in the walking kernel,
  // also the rows' (the epilogue's otherwise) and 1 / s.
  const float* w_scale;
  const float* pair_rows;
  float inv_s;
  // b as int8 rows [k][column]: the scales, b_groups a k, of groups of
  // 2^b_shift columns.
  const float* b_scale;
  int64_t b_groups;
  int b_shift;
  bool b_folded;           // only the scales' powers of two (scale_parts.h): `a` holds the rest
  Epilogue ep;
};

// Kernels: tiles of 256, 128 or 64 rows and columns, or the few-rows kernel on
// 8 rows by 16 columns, 16 by 16 or 32 by 32.
// 8-bit integers have kernels of their own for up to 8 or 16 rows, and for tiles of
// 64 whose operands lie at any address.
enum MatmulTile : int {
  kTile256 = 0, kTile128 = 1, kTile64 = 2, kFew8 = 3, kFew16 = 4, kFew32 = 5, kWalk8 = 6, kWalk16 = 7,
  kAny64 = 8
};

struct MatmulPlan {
  int cfg;
  int splits;
  int64_t ldx, ldw, ldt, ldb;                  // row strides in elements of what the kernel reads
  bool pack_x, pack_w, pack_t, pack_b;         // copied into the workspace at that stride first
  size_t off_x, off_w, off_t, off_b, off_part;
  size_t ws_bytes;
};

// Operand type of the products in 8-bit integers, beside the C ABI's codes.
constexpr int kInt8Operands = 4;
hipError_t gemm_int8(const GemmArgs& g, int out_dtype, int cfg, hipStream_t st);
// The backward's products whose b is int8 rows: tiles of 256 or 128 rows, `a`
// stored [k][row] with a_across.
hipError_t gemm_rows8(const GemmArgs& g, int dtype, bool a_across, int cfg, hipStream_t st);

// The product's plan (dtype: a C ABI code or kInt8Operands, whose t and b are of
// 16 bits); `al` is a bit mask of the operands whose pointers are
// 16-byte aligned (1 x, 2 w, 4 t, 8 b).
MatmulPlan plan_matmul(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int al);

struct MatmulBackwardPlan {
  bool du_direct;                               // du is written into the caller's array alone
  bool direct;                                  // the products read x, w and du in their own layout,
  bool copy;                                    // x and w from copies with a row stride of ldk
  bool x8, w8;                                  // x, w are int8 rows,
  bool x8_tile, w8_tile;                        // read as such by the tile kernel, or brought back into such copies
  bool fold_x, fold_w;                          // their scales, one a row, are in operands of dw and of dx of their own
  bool plain;                                   // du itself is an operand
  int64_t rows;                                 // row blocks of the element-wise pass
  int64_t ldn, ldm, ldk;                        // padded N, M and K
  int cfg_dx, cfg_dw, splits_dx, splits_dw;
  size_t off_du, off_dun, off_dum, off_dut, off_wt, off_xt, off_sum, off_part;
  size_t ws_bytes;
};
// How an operand is held: in the storage type, or as int8 rows with several scales a
// row or one.
enum HeldForm : int { kNotHeld = 0, kHeldGroups = 1, kHeldRows = 2 };
MatmulBackwardPlan plan_matmul_backward(int64_t M, int64_t N, int64_t K, int dtype, bool need_dx, bool need_dw,
                                        bool need_sums, bool du_direct, bool aligned_xw, HeldForm x8, HeldForm w8);

// Operands of the backward that are held as int8 rows (q null: they are not).
struct HeldInt8 {
  Int8Rows u, x, w;
};

// What a backward's products need beside du, in one launch: the element-wise
// pass's partial sums added up (part may be null where there are none), int8 rows
// of w and x in the storage type at a row stride of ldk elements (16 bits), and
// transposed fp32 copies dst[c][r] of src [rows][cols], or of rows8, with zeros up to a row of ld.
struct Turned {
  const void* src;
  Int8Rows rows8;
  int64_t rows, cols, lsrc, ld;
  void* dst;
};
struct BackwardSides {
  bool want_sums;
  const float* part;
  int n_part;
  float* dbias;
  float* dcol;
  Int8Rows w8, x8;
  void* w16;
  void* x16;
  bool w_folded, x_folded;   // by their scales' powers of two alone
  Turned turned[3];
  int n_turned;
  void turn(const void* src, const Int8Rows& r, int64_t rows, int64_t cols, int64_t lsrc, int64_t ld, void* dst) {
    turned[n_turned++] = Turned{src, r, rows, cols, lsrc, ld, dst};
  }
};
hipError_t launch_backward_sides(const BackwardSides& b, int64_t M, int64_t N, int64_t K, int64_t ldk, int dtype,
                                 hipStream_t st);

hipError_t launch_matmul(const MatmulPlan& p, const void* x, const void* w, int dtype, int64_t M, int64_t N,
                         int64_t K, const void* t, const void* b, int64_t r, float s, const Epilogue& ep,
                         const float* w_scale, int out_dtype, char* ws, hipStream_t st);
hipError_t launch_matmul_backward(const MatmulBackwardPlan& p, const void* dy, const void* u, const void* x,
                                  const void* w, int dtype, int64_t M, int64_t N, int64_t K, const float* row_scale,
                                  const float* col_scale, const float* bias, int act, void* du, void* dx, void* dw,
                                  float* dbias, float* dcol, const HeldInt8& held, char* ws, hipStream_t st);

}  // namespace dora
