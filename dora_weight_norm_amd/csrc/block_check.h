// Argument checks shared by the C entry points of the block's operators (host side).
#pragma once

#include <math.h>

#include "dora_check.h"
#include "dora_matmul.h"

namespace dora {

// One buffer of a call: its bytes, and the alignment its elements need.
struct Span {
  const void* p;
  int64_t bytes;
  size_t align;
};

// Every element of a tensor is reached with 64-bit arithmetic far from its
// limits, and every launch stays within its grid.
constexpr int64_t kMaxElems = (int64_t)1 << 33;
// Bytes of one row of a product's operand (the tile kernel's 32-bit offsets
// span 256 rows).
constexpr int64_t kMaxRowBytes = (int64_t)1 << 23;
// Rows of a product: 64 of them a workgroup of 256 threads, and a launch takes
// less than 2^32 threads.
constexpr int64_t kMaxRows = (int64_t)1 << 30;

inline bool size_ok(int64_t a, int64_t b) {
  return a >= 0 && b >= 0 && a < kMaxDim && b < kMaxDim && (b == 0 || a <= kMaxElems / b);
}

// Inputs and outputs are aligned; no output overlaps an input or another
// output, except input i that output o may be exactly (bit i of same[o]).
inline bool buffers_ok(const Span* in, int n_in, const Span* out, int n_out, const unsigned* same) {
  for (int i = 0; i < n_in; ++i)
    if (!aligned(in[i].p, in[i].align)) return false;
  for (int o = 0; o < n_out; ++o) {
    if (!aligned(out[o].p, out[o].align)) return false;
    for (int i = 0; i < n_in; ++i) {
      if ((same[o] >> i & 1u) && out[o].p == in[i].p) continue;
      if (overlap(out[o].p, out[o].bytes, in[i].p, in[i].bytes)) return false;
    }
    for (int q = o + 1; q < n_out; ++q)
      if (overlap(out[o].p, out[o].bytes, out[q].p, out[q].bytes)) return false;
  }
  return true;
}

inline dora_status workspace_ok(const void* ws, size_t have, size_t need, const Span* in, int n_in, const Span* out,
                         int n_out) {
  if (need == 0) return DORA_OK;
  if (have < need || ws == nullptr || !aligned(ws, kAlign)) return DORA_ERR_WORKSPACE;
  for (int i = 0; i < n_in; ++i)
    if (overlap(ws, (int64_t)need, in[i].p, in[i].bytes)) return DORA_ERR_INVALID_ARG;
  for (int o = 0; o < n_out; ++o)
    if (overlap(ws, (int64_t)need, out[o].p, out[o].bytes)) return DORA_ERR_INVALID_ARG;
  return DORA_OK;
}

inline bool valid_act(int act) { return act >= DORA_ACT_NONE && act <= DORA_ACT_SILU; }
inline int64_t operand_size(int dt) { return dt == DORA_E4M3 ? 1 : esize(dt); }

inline bool matmul_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t r, int64_t es) {
  return size_ok(M, K) && size_ok(N, K) && size_ok(M, N) && size_ok(M, r) && size_ok(N, r) &&
         M < kMaxRows && K * es < kMaxRowBytes && r * es < kMaxRowBytes && N < kMaxRowBytes;
}

// The backward's products run along M and N too.
inline bool backward_sizes_ok(int64_t M, int64_t N, int64_t K, int64_t es) {
  return matmul_sizes_ok(M, N, K, 0, es) && M * es < kMaxRowBytes && N * es < kMaxRowBytes;
}

// Rows of a tile; 0 for the kernels of few rows.
inline int plan_tile_rows(int cfg) {
  return cfg == kTile256 ? 256 : (cfg == kTile128 ? 128 : (cfg == kTile64 || cfg == kAny64 ? 64 : 0));
}

// A product's plan as its query gives it.
inline void plan_fields(const MatmulPlan& p, bool any, bool int8, int64_t* info, int n_info) {
  const int copies = (p.pack_x ? 1 : 0) | (p.pack_w ? 2 : 0) | (p.pack_t ? 4 : 0) | (p.pack_b ? 8 : 0);
  const int few = p.cfg == kFew8 || p.cfg == kWalk8 ? 8
                  : (p.cfg == kFew16 || p.cfg == kWalk16 ? 16 : (p.cfg == kFew32 ? 32 : -1));
  const int kernel = p.cfg < kFew8 ? 0 : (p.cfg == kAny64 ? 3 : (p.cfg == kWalk8 || p.cfg == kWalk16 ? 2 : 1));
  const int64_t vals[] = {any ? plan_tile_rows(p.cfg) : -1, p.splits, copies, (int64_t)p.ws_bytes, few,
                          any && int8 ? kernel : -1};
  for (int i = 0; i < n_info; ++i) info[i] = i < 6 ? vals[i] : -1;
}

}  // namespace dora
