// How 256 threads walk rows held in 8-bit integers, and such rows brought back to
// a storage type.
#pragma once

#include "dora_launch.h"
#include "dora_rows.h"
#include "scale_parts.h"

namespace dora {

namespace {

// 256 threads are 2^lanes of them along a row by 2^(8 - lanes) rows; an item is
// one such step, `steps` of them along a row. kItems items' loads are in flight at
// a time.
constexpr int kItems = 2;
constexpr int64_t kMostGroups = 65536;   // of 256 threads

struct RowSteps {
  int64_t T, d;
  int64_t groups;      // scales a row
  int shift;           // log2 of the columns of a group (group_shift)
  int lanes;
  uint32_t steps, items;
};

struct Place {
  int64_t row, k;      // row, and first column
  bool ok;
};

// Of thread t of the 256.
template <int E>
__device__ __forceinline__ Place place_of(const RowSteps& s, uint32_t item, uint32_t t) {
  const uint32_t r = item / s.steps, c = item - r * s.steps;   // (uniform)
  Place p;
  p.row = ((int64_t)r << (8 - s.lanes)) + (t >> s.lanes);
  p.k = (((int64_t)c << s.lanes) + (t & ((1u << s.lanes) - 1))) * E;
  p.ok = item < s.items && p.row < s.T && p.k < s.d;
  return p;
}

// One or two operands of rows of d columns, the second's rows numbered after the
// first's; rows of x lie ld >= d elements apart, and those from d on, up to a
// whole chunk or ld, are written as zeros. A value is the fp32 product of q and its
// scale, rounded once to T (as the tile kernel rounds rows that it reads as they are
// held: a product's operands have 16 bits), or with its power of two alone where FOLD
// and the job say so, which is exact.
struct UnpackJob {
  const uint8_t* q;
  const float* scale;
  int64_t groups, T;
  int shift;
  void* x;
  bool folded;
};

// Thread t of the 256 that are number `group` of `groups`.
template <typename T, bool STREAM, bool FOLD>
__device__ __forceinline__ void unpack_rows(const UnpackJob& a, const UnpackJob& b, const RowSteps& s, int64_t ld,
                                            uint32_t group, uint32_t groups, uint32_t t) {
  constexpr int E = Elem<T>::epc;
  for (uint32_t it = group * kItems; it < s.items; it += groups * kItems) {
    uint32_t w[kItems][E / 4];
    float sc[kItems];
    Place p[kItems];
    T* to[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      p[i] = place_of<E>(s, it + i, t);
      const bool first = p[i].row < a.T;
      const int64_t row = first ? p[i].row : p[i].row - a.T;
      to[i] = static_cast<T*>(first ? a.x : b.x) + row * ld;
      if (p[i].ok) {
        load_row_bytes<E>((first ? a.q : b.q) + row * s.d, p[i].k, s.d, w[i]);
        sc[i] = (first ? a.scale : b.scale)[row * (first ? a.groups : b.groups) + (p[i].k >> (first ? a.shift : b.shift))];
      }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (!p[i].ok) continue;
      if constexpr (FOLD) sc[i] = FoldBits<T>(p[i].row < a.T ? a.folded : b.folded)(sc[i]);
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = (float)(int8_t)(w[i][e / 4] >> (8 * (e % 4))) * sc[i];
      store_row_chunk<T, STREAM>(to[i], p[i].k, ld, f);
    }
  }
}

// The steps of rows whose chunks of E elements are padded to whole groups of L.
[[maybe_unused]] RowSteps row_steps(int64_t T, int64_t d, int64_t group, int E, int L) {
  RowSteps s{};
  s.T = T, s.d = d;
  s.groups = scales_of(d, group);
  s.shift = group_shift(group);
  const int64_t chunks = ((d + E - 1) / E + L - 1) / L * L;
  while (s.lanes < 8 && ((int64_t)1 << s.lanes) < chunks) ++s.lanes;
  const int64_t by = 256 >> s.lanes;
  s.steps = (uint32_t)((chunks + (1 << s.lanes) - 1) >> s.lanes);
  s.items = (uint32_t)((T + by - 1) / by * s.steps);
  return s;
}

// Groups of 256 threads that take them.
[[maybe_unused]] unsigned row_groups(const RowSteps& s) {
  const int64_t groups = ((int64_t)s.items + kItems - 1) / kItems;
  return (unsigned)(groups < kMostGroups ? groups : kMostGroups);
}

[[maybe_unused]] UnpackJob unpack_job(const Int8Rows& r, int64_t T, int64_t d, void* x, bool folded) {
  return UnpackJob{r.q, r.scale, scales_of(d, r.group), T, group_shift(r.group), x, folded};
}

}  // namespace

}  // namespace dora
