// Kernels of the matrix products and their launches, for the files that instantiate them.
#pragma once

#include "dora_device.h"
#include "dora_launch.h"
#include "dora_matmul.h"
#include "scale_parts.h"

namespace dora {

namespace {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct e4m3_t {
  uint8_t v;
};
struct int8x_t {   // 8-bit integers
  int8_t v;
};
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// Operand types: bytes of an element, 16-byte chunks of a lane's fragment,
// and one matrix instruction step over 2 * FC chunks of depth.
template <typename T>
struct Op;
template <>
struct Op<bf16_t> {
  static constexpr int esz = 2, fc = 1;
  static __device__ __forceinline__ f32x16 run(const u32x4* a, const u32x4* b, f32x16 c) {
    return Mfma<bf16_t>::run(a, b, c);
  }
};
template <>
struct Op<f16_t> {
  static constexpr int esz = 2, fc = 1;
  static __device__ __forceinline__ f32x16 run(const u32x4* a, const u32x4* b, f32x16 c) {
    return Mfma<f16_t>::run(a, b, c);
  }
};
template <>
struct Op<float> {
  static constexpr int esz = 4, fc = 2;
  static __device__ __forceinline__ f32x16 run(const u32x4* a, const u32x4* b, f32x16 c) {
    return Mfma<float>::run(a, b, c);
  }
};
template <>
struct Op<e4m3_t> {
  static constexpr int esz = 1, fc = 2;
  // v_mfma_scale_f32_32x32x64_f8f6f4 on two e4m3 operands, all block scales
  // 2^0 (exponent byte 127). gfx950's 8-bit matrix instructions, all of them,
  // align each group of eight products to the largest and drop what lies
  // 2^-13 below it (found with directed in-bounds probes); the sums over the
  // groups and the accumulators are fp32. Exact sums would take the bf16
  // instructions at half the rate; on normal data the loss is 2^-17 of the
  // sum of sizes, far below the operands' own 2^-4 steps.
  static __device__ __forceinline__ f32x16 run(const u32x4* a, const u32x4* b, f32x16 c) {
    struct P {
      u32x4 lo, hi;
    };
    const P pa{a[0], a[1]}, pb{b[0], b[1]};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(__builtin_bit_cast(i32x8, pa), __builtin_bit_cast(i32x8, pb),
                                                           c, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
  }
};

template <>
struct Op<int8x_t> {
  static constexpr int esz = 1, fc = 1;
  // Integer sums, in the registers that hold fp32 ones elsewhere (0 has the
  // same bits in both).
  static __device__ __forceinline__ f32x16 run(const u32x4* a, const u32x4* b, f32x16 c) {
    return __builtin_bit_cast(f32x16, __builtin_amdgcn_mfma_i32_32x32x32_i8(
                                          __builtin_bit_cast(i32x4, a[0]), __builtin_bit_cast(i32x4, b[0]),
                                          __builtin_bit_cast(i32x16, c), 0, 0, 0));
  }
};

// The low-rank pair's type: the operands' own, but 16 bits, the output's,
// beside 8-bit integers.
template <typename T, typename O>
struct PairType {
  using type = T;
};
template <typename O>
struct PairType<int8x_t, O> {
  using type = std::conditional_t<sizeof(O) == 2, O, bf16_t>;   // (fp32 outputs come without a pair)
};

// Activations (dora_act) and their slopes, in fp32 arithmetic. F32: the result
// is stored in fp32, and the device library's exponential, error function and
// division are used, whose errors are a step or two of it (2048^3 with GELU:
// 144 us, 140 with the forms below). Results of 16 bits take the forms below,
// whose errors relative to the result are far below half of their steps
// (2^-11 in fp16) in the tails too.
constexpr float kTanhK = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kTanhC = 0.044715f;

// 1 / (1 + e^-v). 16 bits: by the hardware's exponential of base two and
// reciprocal (one unit in the last place each; the product with log2(e) adds
// |v| 2^-23 relative): a correctly rounded division and expf cost the epilogue
// of the 8192 x 28672 product about as much again as its stores.
template <bool F32>
__device__ __forceinline__ float logistic(float v) {
  if constexpr (F32) return 1.f / (1.f + expf(-v));
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896f * v));
}

// Phi(z) = erfc(-z / sqrt 2) / 2. 16 bits: with x = |z| / sqrt 2 and t = 1 / (1 +
// p x), erfc(x) = (a1 t + ... + a8 t^8) e^(-x^2), a fit of e^(x^2) erfc(x) in
// the relative error, at most 1.1e-7 for x up to 11 (found by weighted least
// squares); with fp32's roundings (16 + 2 z^2) 2^-24 of Phi, a few steps of
// fp32 where the tail matters. Results below 2^-126 may be 0.
template <bool F32>
__device__ __forceinline__ float normal_cdf(float z) {
  if constexpr (F32) return 0.5f * erfcf(z * -0.70710678118654752f);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.332f * 0.70710678118654752f, fabsf(z), 1.f));
  float q = fmaf(t, -0.129304167f, 0.42600419f);
  q = fmaf(t, q, -0.29990073f);
  q = fmaf(t, q, 0.366505857f);
  q = fmaf(t, q, 0.067685469f);
  q = fmaf(t, q, 0.196667373f);
  q = fmaf(t, q, 0.184907024f);
  q = fmaf(t, q, 0.187434877f);
  const float h = 0.5f * (q * t) * __builtin_amdgcn_exp2f(-0.72134752044448f * (z * z));   // erfc(x) / 2
  return z < 0.f ? h : 1.f - h;
}

template <bool F32>
__device__ __forceinline__ float act1(float z, int act) {
  switch (act) {
    case 1: return z < 0.f ? 0.f : z;
    case 2: return z * normal_cdf<F32>(z);
    // z / 2 (1 + tanh(v)) = z / (1 + exp(-2 v))
    case 3: return z * logistic<F32>(z * fmaf(2.f * kTanhK * kTanhC, z * z, 2.f * kTanhK));
    case 4: return z * logistic<F32>(z);
    default: return z;
  }
}

// N values at once, so that the (uniform) choice is made once.
template <int N, bool F32>
__device__ __forceinline__ void act_all(float (&z)[N], int act) {
  switch (act) {
#define DORA_ACT(A)                                           \
  case A:                                                     \
    for (int e = 0; e < N; ++e) z[e] = act1<F32>(z[e], A);    \
    break;
    DORA_ACT(1)
    DORA_ACT(2)
    DORA_ACT(3)
    DORA_ACT(4)
#undef DORA_ACT
    default: break;
  }
}

template <bool F32>
__device__ __forceinline__ float slope_of(float z, int act) {
  switch (act) {
    case 1: return z > 0.f ? 1.f : (z != z ? z : 0.f);
    case 2: {
      const float e = -0.72134752044448f * (z * z);   // e^(-z^2 / 2) = 2^e
      return normal_cdf<F32>(z) + z * 0.3989422804014327f * (F32 ? exp2f(e) : __builtin_amdgcn_exp2f(e));
    }
    case 3: {
      const float p = logistic<F32>(z * fmaf(2.f * kTanhK * kTanhC, z * z, 2.f * kTanhK));
      // (past 32 p is 0 or 1 and the other term 0: z^2 may be infinite there)
      const float c = fminf(fmaxf(z, -32.f), 32.f);
      return p + c * p * (1.f - p) * 2.f * kTanhK * fmaf(3.f * kTanhC * c, c, 1.f);
    }
    case 4: {
      const float p = logistic<F32>(z);
      return p * (1.f + z * (1.f - p));
    }
    default: return 1.f;
  }
}

// z to the activation's slope there, N values at once.
template <int N, bool F32>
__device__ __forceinline__ void slope_all(float (&z)[N], int act) {
  switch (act) {
#define DORA_SLOPE(A)                                           \
  case A:                                                       \
    for (int e = 0; e < N; ++e) z[e] = slope_of<F32>(z[e], A);  \
    break;
    DORA_SLOPE(0)
    DORA_SLOPE(1)
    DORA_SLOPE(2)
    DORA_SLOPE(3)
    DORA_SLOPE(4)
#undef DORA_SLOPE
    default: break;
  }
}

// Eight consecutive elements of an output row in the output type, as loaded.
template <typename O>
struct Raw8 {
  u32x4 v[8 / Elem<O>::epc];
};

template <typename O, bool STREAM = false>
__device__ __forceinline__ Raw8<O> load_raw8(const O* p, int n) {
  constexpr int E = Elem<O>::epc;
  Raw8<O> r;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < 8 / E; ++i) {
      const u32x4_any* q = reinterpret_cast<const u32x4_any*>(p + i * E);
      if constexpr (STREAM)
        r.v[i] = __builtin_nontemporal_load(q);
      else
        r.v[i] = *q;
    }
  } else {
    O tmp[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) tmp[e] = e < n ? p[e] : O(0);
    __builtin_memcpy(&r, tmp, sizeof(r));
  }
  return r;
}

template <typename O>
__device__ __forceinline__ void unpack8(const Raw8<O>& r, float (&f)[8]) {
  constexpr int E = Elem<O>::epc;
#pragma unroll
  for (int i = 0; i < 8 / E; ++i) {
    float g[E];
    unpack<O, E>(r.v[i], g);
#pragma unroll
    for (int e = 0; e < E; ++e) f[i * E + e] = g[e];
  }
}

template <typename O>
__device__ __forceinline__ void load8(const O* p, int n, float (&f)[8]) {
  unpack8<O>(load_raw8<O>(p, n), f);
}

template <typename O>
__device__ __forceinline__ void store8(O* p, int n, const float (&f)[8]) {
  constexpr int E = Elem<O>::epc;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < 8 / E; ++i) {
      float g[E];
#pragma unroll
      for (int e = 0; e < E; ++e) g[e] = f[i * E + e];
      *reinterpret_cast<u32x4_any*>(p + i * E) = pack<O, E>(g);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = from_f32<O>(f[e]);
  }
}

// The epilogue on eight consecutive columns of R rows: row m[i] at offset
// off[i] if ok[i]; cs and bs are the columns' scales and biases, n how many of
// them exist, res the rows' residual (already loaded).
template <typename O, int R>
__device__ __forceinline__ void epilogue_rows(const Epilogue& ep, float (&v)[8 * R], const float (&cs)[8],
                                              const float (&bs)[8], const int64_t (&m)[R], const int64_t (&off)[R],
                                              const bool (&ok)[R], int n, const Raw8<O> (&res)[R]) {
  if (ep.row_scale) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float rs = ok[i] ? ep.row_scale[m[i]] : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] *= rs;
    }
  }
  auto put = [&](void* to) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = v[8 * i + e];
      if (ok[i]) store8<O>(static_cast<O*>(to) + off[i], n, o);
    }
  };
  if (ep.u) put(ep.u);
#pragma unroll
  for (int e = 0; e < 8 * R; ++e) v[e] = fmaf(cs[e % 8], v[e], bs[e % 8]);
  act_all<8 * R, std::is_same<O, float>::value>(v, ep.act);
  if (ep.residual) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float r[8];
      unpack8<O>(res[i], r);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] += r[e];
    }
  }
  put(ep.y);
}

// The epilogue on one element.
template <typename O>
__device__ __forceinline__ void epilogue1(const Epilogue& ep, float v, float cs, float bs, int64_t m, int64_t off) {
  if (ep.row_scale) v *= ep.row_scale[m];
  if (ep.u) static_cast<O*>(ep.u)[off] = from_f32<O>(v);
  v = act1<std::is_same<O, float>::value>(fmaf(cs, v, bs), ep.act);
  if (ep.residual) v += to_f32(static_cast<const O*>(ep.residual)[off]);
  static_cast<O*>(ep.y)[off] = from_f32<O>(v);
}

// Eight column scales and biases from column c on, n of them there.
__device__ __forceinline__ void column_terms(const Epilogue& ep, int64_t c, int n, float (&cs)[8], float (&bs)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) cs[e] = 1.f, bs[e] = 0.f;
  if (n <= 0) return;
  if (ep.col_scale) load8<float>(ep.col_scale + c, n, cs);
  if (ep.bias) load8<float>(ep.bias + c, n, bs);
}

// One operand's share of a stage, R rows by 128 bytes of depth, staged in LDS
// by direct loads of 1 KiB (64 lanes x 16 bytes). Wave w of NW makes loads w,
// w + NW, ...; a lane's offset in its load b is off + b * step.
//   Rows along the depth ([row][k] in memory): an LDS row is one row's 128
// bytes, a load eight of them; chunk c of row r lies at chunk c ^ (r / 2 mod
// 8). Rows past the operand lie past the descriptor's end and read zeros.
//   TR, rows across it ([k][row] in memory, 16-bit types): an LDS row is one
// k's R elements, 64 of them a stage; chunk c of k lies at c ^ trswz(k), under
// which the four k that a transposing read touches at once lie in distinct
// banks. Columns past the operand are out of range per lane, and k past the
// depth lie past the descriptor's end.
template <int R>
__device__ __forceinline__ int trswz(int k) {
  return R >= 128 ? (k & 3) << 2 : ((k >> 1) & 1) << 2;
}

struct Stream {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off, step;
  const char* p;      // TR: the operand, and bytes of one k
  int64_t kbytes;
};

template <int ESZ, int R, int NW, bool TR>
__device__ __forceinline__ Stream make_stream(const void* p, int64_t ld, int64_t row0, int64_t rows, int lane,
                                              int wave) {
  Stream s;
  s.p = static_cast<const char*>(p);
  s.kbytes = ld * ESZ;
  if constexpr (TR) {
    constexpr int CPR = R / 8, KPB = 64 / CPR;   // chunks of an LDS row, k a load
    const int k = wave * KPB + lane / CPR;
    const int64_t col = row0 + ((lane % CPR) ^ trswz<R>(k)) * 8;
    s.rsrc = make_rsrc(p, 0u);
    s.off = col < rows ? (uint32_t)(k * s.kbytes + col * ESZ) : kOob;
    s.step = (uint32_t)(NW * KPB * s.kbytes);
  } else {
    const int64_t left = rows - row0 < R ? rows - row0 : R;
    const int chunk = (lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7);
    s.rsrc = make_rsrc(s.p + row0 * s.kbytes, p ? (uint32_t)(left * s.kbytes) : 0u);
    s.off = (uint32_t)((wave * 8 + (lane >> 3)) * s.kbytes) + (uint32_t)(chunk * 16);
    s.step = (uint32_t)(NW * 8 * s.kbytes);
  }
  return s;
}

// A lane's fragment (row r0 + lane % 32, eight k of step s from 8 (lane / 32))
// of an operand staged as [k][R rows]: two transposing reads, each of which
// gives lane i of 16 four k of row i from the rows of four k that its group's
// lanes point at.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// (A function of its own with a restricted pointer: inlining it gives the read
// alias information. Without any, the compiler takes it to depend on every
// direct load in flight and waits for them all.)
__device__ __forceinline__ s16x4 tr_load(lds_s16x4* __restrict p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16(p); }

// Two values as 16-bit ones, round to nearest even.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
  const f32x2 v = {a, b};
  if constexpr (std::is_same<T, bf16_t>::value) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// (likewise)
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
__device__ __forceinline__ void store_lds(lds_u32x4* __restrict p, u32x4 v) { *p = v; }

template <int R>
__device__ __forceinline__ u32x4 read_tr(const char* unit, int r0, int s, int lane) {
  const int g = lane >> 4, m = lane & 15;
  const int col = r0 + 16 * (g & 1) + 4 * (m & 3);
  s16x4 h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = s * 16 + 8 * (g >> 1) + 4 * i + (m >> 2);
    const char* at = unit + k * (R * 2) + (((col >> 3) ^ trswz<R>(k)) * 16 + (col & 7) * 2);
    h[i] = tr_load((lds_s16x4*)at);
  }
  struct P {
    s16x4 lo, hi;
  };
  const P p{h[0], h[1]};
  return __builtin_bit_cast(u32x4, p);
}

// ---------------------------------------------------------------------------
// Tile kernel. Workgroup = WM x WN waves = one tile of (WM MB 32) rows by
// (WN NB 32) columns over one part of the depth. A stage is 128 bytes of depth
// of both operands. LDS holds a ring of 2P + 1 units of one operand's stage:
// stage i's rows are in unit 2i and its columns in unit 2i + 1 (mod 2P + 1).
// With the stages up to i + P - 1 and the rows of stage i + P already there,
// the two units that stage i frees take the columns of stage i + P first and
// the rows of stage i + P + 1 after them. At P = 2, which fills LDS for the
// 256-row tile, half of the loads so have a whole stage to land and half have
// two (8192^3 bf16: 806 us, against 860 us with two slots of whole stages and
// the next lines asked into L2 ahead); the 64-row tile takes P = 4. One
// barrier a stage, where a wave has read all of stage i; a wave holds two sets
// of fragments and reads the next step's while this step's matrix instructions
// run.
// ---------------------------------------------------------------------------
// B8: the columns are int8 rows [k][column] with a scale for each k and group of
// columns, brought to the 16-bit type on their way to LDS. A lane takes 16
// bytes of a k at a time, loaded one period ahead, and converts and stores them
// element by element between the period's matrix instructions: each element of
// the stage once a workgroup, where a conversion behind the transposing reads
// would do it in every wave. A value q times its scale is rounded to 16 bits there,
// half a step of 2^-8 (2^-11) of it: a scale of a group of columns differs from one
// k to the next and from one column to another, so that no factor of a row, a column
// or the result can take it. Of one scale a row the other operand holds the
// significand (b_folded), and the integer times a power of two is exact.
template <typename T, typename O, int WM, int WN, int MB, int NB, int P, bool PAIR, bool AT, bool BT, bool B8 = false>
__global__ __launch_bounds__(WM* WN * 64, 1) void matmul_tile_kernel(GemmArgs g) {
  constexpr int ESZ = Op<T>::esz, FC = Op<T>::fc, KT = 128 / ESZ;
  constexpr int NW = WM * WN, MT = WM * MB * 32, NT = WN * NB * 32;
  constexpr int UNIT = (MT > NT ? MT : NT) * 128;           // bytes of a ring unit
  // 1 KiB blocks per wave per stage (B8: 16 bytes a lane, which become 32)
  constexpr int ABLK = MT / 8 / NW, BBLK = NT / (B8 ? 16 : 8) / NW;
  constexpr int BPW = ABLK + BBLK;
  constexpr int STEPS = 8 / (2 * FC);
  // 8-bit integers: their sums come first, are converted and scaled in the
  // registers, and the pair's products are added to them there.
  constexpr bool I8 = std::is_same<T, int8x_t>::value;
  using TP = typename PairType<T, O>::type;
  constexpr int ESZ2 = Op<TP>::esz, KT2 = 128 / ESZ2;
  static_assert(Op<TP>::fc == FC, "the pair's stages have as many steps");
  constexpr int EPW = NB * 32 + 4;                         // floats of an epilogue row (padded: no bank conflicts)
  static_assert(MT % (8 * NW) == 0 && NT % (8 * NW) == 0, "a stage splits evenly over the waves");
  constexpr int RING = (2 * P + 1) * UNIT;
  static_assert((NW * 32 * EPW + (I8 ? NW * NB * 32 : 0)) * 4 <= RING, "the epilogue fits the ring");
  static_assert(RING <= 160 * 1024, "gfx950 has 160 KiB of LDS");
  static_assert(STEPS % 2 == 0, "step s of every stage uses fragment set s & 1");
  extern __shared__ __align__(1024) char lds[];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // Workgroup i runs on die i % 8: each die takes a contiguous run of tiles,
  // in groups of eight row tiles by all column tiles, so that the tiles on
  // one die at one time share their operands in its L2.
  const int total = g.n_mt * g.n_nt;
  int id = blockIdx.x;
  const int split = id / total;
  id -= split * total;
  {
    const int q = total / 8, r = total % 8, x = id % 8;
    id = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + id / 8;
  }
  const int gsz = 8 * g.n_nt, grp = id / gsz, first = grp * 8;
  const int gm = g.n_mt - first < 8 ? g.n_mt - first : 8;
  const int mt = first + (id - grp * gsz) % gm, nt = (id - grp * gsz) / gm;
  const int64_t m0 = (int64_t)mt * MT, n0 = (int64_t)nt * NT;

  const int chunk = (lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7);   // of depth, in rows along it
  const Stream sa = make_stream<ESZ, MT, NW, AT>(g.a, g.lda, m0, g.M, lane, wave);
  const Stream sb = make_stream<ESZ, NT, NW, BT>(g.b, g.ldb, n0, g.N, lane, wave);
  const Stream sa2 = make_stream<ESZ2, MT, NW, false>(g.a2, g.lda2, m0, g.M, lane, wave);
  const Stream sb2 = make_stream<ESZ2, NT, NW, false>(g.b2, g.ldb2, n0, g.N, lane, wave);
  // Stages: the low-rank pair's first, then the main depth's (8-bit integers:
  // the other way round); this workgroup's part of them is [st0, st1).
  const int n2 = PAIR ? (int)((g.K2 + KT2 - 1) / KT2) : 0;
  const int n1 = I8 ? (int)((g.K + KT - 1) / KT) : 0;
  const int st0 = split * g.stages_per_split;
  const int st1 = st0 + g.stages_per_split < g.stages ? st0 + g.stages_per_split : g.stages;

  // Load b of one operand's stage i into a ring unit. Past the depth every
  // lane's offset is out of range (zeros), so that every stage issues the same
  // loads. (Arguments are named before the builtin: a conditional inside its
  // argument list makes the host pass drop the kernel's stub.)
  auto issue = [&](const Stream& main, const Stream& pair, int i, int unit, int b, auto tr)
      __attribute__((always_inline)) {
    char* dst = lds + unit + (b * NW + wave) * 1024;
    if constexpr (decltype(tr)::value) {
      const int64_t left = (i < st1 ? g.K - (int64_t)i * KT : 0) * main.kbytes;
      const uint32_t bytes = (uint32_t)(left < 0 ? 0 : (left < 0x7fffffff ? left : 0x7fffffff));
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(main.p + (int64_t)i * KT * main.kbytes, bytes);
      const uint32_t off = main.off + (uint32_t)b * main.step;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
    } else {
      const bool pr = PAIR && (I8 ? i >= n1 : i < n2);
      const int k0 = (I8 ? (pr ? i - n1 : i) : (pr ? i : i - n2)) * 128;   // bytes of depth before the stage
      const int left = i < st1 ? (int)(pr ? g.K2 * ESZ2 : g.K * ESZ) - k0 : 0;
      const uint32_t at = pr ? pair.off + (uint32_t)b * pair.step : main.off + (uint32_t)b * main.step;
      const uint32_t off = chunk * 16 < left ? at : kOob;
      const __amdgpu_buffer_rsrc_t rs = pr ? pair.rsrc : main.rsrc;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, k0, 0, 0);
    }
  };
  // B8: a lane's 16 bytes j are those of k (wave * 64 + lane) / CPK + j * KPJ and
  // of column 16 ((lane) % CPK) of the tile.
  constexpr int CPK = NT / 16, KPJ = NW * 64 / CPK, PER_STEP = BBLK * 16 / STEPS;
  static_assert(!B8 || (BT && !PAIR && ESZ == 2 && P == 2 && BBLK * KPJ == 64 && (PER_STEP == 16 || PER_STEP == 8)),
                "a step converts one or half of a lane's 16 bytes");
  u32x4 qv[B8 ? BBLK : 1], qout = {0u, 0u, 0u, 0u};
  float qs[B8 ? BBLK : 1];
  const int qk = (int)threadIdx.x / CPK, qc = (int)threadIdx.x % CPK;
  const bool q_in = n0 + qc * 16 < g.N;   // (rows are whole chunks)
  const uint32_t q_off = q_in ? (uint32_t)(qk * g.ldb + n0 + qc * 16) : kOob;
  const uint32_t s_off = (uint32_t)(qk * g.b_groups + ((n0 + qc * 16) >> g.b_shift)) * 4u;
  // The stage that is being loaded, as addresses and bytes up to the end of this
  // workgroup's depth, which advance by a stage at a time (computed anew for each
  // load they were a third of the loop's instructions, of which one wave a SIMD
  // issues one in four cycles).
  const int64_t k_end = g.K < (int64_t)st1 * 64 ? g.K : (int64_t)st1 * 64, k_first = k_end - (int64_t)st0 * 64;
  const char* q_at = static_cast<const char*>(g.b) + (int64_t)st0 * 64 * g.ldb;
  const char* s_at = reinterpret_cast<const char*>(g.b_scale) + (int64_t)st0 * 256 * g.b_groups;
  const char* a_at = sa.p + (int64_t)st0 * 64 * sa.kbytes;
  int64_t q_left = k_first * g.ldb, s_left = k_first * g.b_groups * 4, a_left = k_first * sa.kbytes;
  auto bytes = [](int64_t left) __attribute__((always_inline)) {
    return (uint32_t)(left < 0 ? 0 : (left < 0x7fffffff ? left : 0x7fffffff));
  };
  uint32_t q_bytes = bytes(q_left), s_bytes = bytes(s_left), a_bytes = bytes(a_left);
  auto advance = [&]() __attribute__((always_inline)) {
    q_at += 64 * g.ldb, s_at += 256 * g.b_groups, a_at += 64 * sa.kbytes;
    q_left -= 64 * g.ldb, s_left -= 256 * g.b_groups, a_left -= 64 * sa.kbytes;
    q_bytes = bytes(q_left), s_bytes = bytes(s_left), a_bytes = bytes(a_left);
  };
  auto load_q = [&](int j) __attribute__((always_inline)) {
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(q_at, q_bytes), rs = make_rsrc(s_at, s_bytes);
    const uint32_t qo = q_off + (uint32_t)(j * KPJ) * (uint32_t)g.ldb;
    const uint32_t so = s_off + (uint32_t)(j * KPJ) * (uint32_t)g.b_groups * 4u;
    qv[j] = __builtin_amdgcn_raw_buffer_load_b128(rq, qo, 0, 0);
    qs[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, so, 0, 0));
  };
  // Element e of the stage's BBLK * 16 of this lane, into the unit; with the last
  // of 16 bytes the next stage's take their registers.
  float qf = 0.f;
  const FoldBits<T> fold(B8 && g.b_folded);
  auto convert = [&](int unit, int e) __attribute__((always_inline)) {
    if constexpr (B8) {
      const int j = e / 16, b = e % 16;
      // (bytes that a later step takes are not to be picked out, and so waited for,
      // when they were only just asked for)
      if (b % 8 == 0) asm volatile("" : "+v"(qv[j]), "+v"(qs[j]));
      if (b == 0) qs[j] = fold(qs[j]);
      const float f = (float)(int8_t)(qv[j][b / 4] >> (8 * (b % 4))) * qs[j];
      if (b % 2)
        qout[b % 8 / 2] = pack2<T>(qf, f);
      else
        qf = f;
      if (b % 8 == 7) {
        const int k = qk + j * KPJ, c = qc * 2 + b / 8;
        store_lds((lds_u32x4*)(lds + unit + k * (NT * 2) + ((c ^ trswz<NT>(k)) * 16)), qout);
      }
      if (b == 15) load_q(j);
    }
  };
  auto issue_a = [&](int i, int unit, int b) __attribute__((always_inline)) { issue(sa, sa2, i, unit, b, Tag<AT>{}); };
  // (B8: of the stage being loaded, whose number i is.)
  auto issue_a8 = [&](int i, int unit, int b) __attribute__((always_inline)) {
    if constexpr (AT) {
      char* dst = lds + unit + (b * NW + wave) * 1024;
      const __amdgpu_buffer_rsrc_t rs = make_rsrc(a_at, a_bytes);
      const uint32_t off = sa.off + (uint32_t)b * sa.step;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, 0);
    } else {
      issue_a(i, unit, b);
    }
  };
  auto issue_b = [&](int i, int unit, int b) __attribute__((always_inline)) { issue(sb, sb2, i, unit, b, Tag<BT>{}); };

  // The epilogue's columns of this lane: their scales and biases are asked for
  // here, a whole depth before they are needed.
  constexpr int LPR = NB * 4, RPP = 64 / LPR, PB = 32 / RPP;   // lanes a row, rows a pass, passes a block
  const int col = (lane % LPR) * 8;
  const int64_t n = n0 + wn * NB * 32 + col;
  const int nv = (int)(g.N - n < 8 ? g.N - n : 8);
  float cs[8], bs[8];
  if constexpr (!B8) column_terms(g.ep, n, nv, cs, bs);   // (B8: a product of the backward, stored as it is or times a row's scale)
  f32x16 acc[MB][NB];
#pragma unroll
  for (int a = 0; a < MB; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.f;

  const int fr = lane & 31, fg = lane >> 5;
  struct Frag {
    u32x4 a[MB][FC], b[NB][FC];
  };
  // Read q of a step's (MB + NB) FC fragment pieces, in the order in which the
  // step's matrix instructions (row blocks outermost) come to need them: the
  // first row block, the column blocks, the other row blocks.
  constexpr int ND = (MB + NB) * FC, NM = MB * NB;
  auto read = [&](int ua, int ub, int s, Frag& F, int q) __attribute__((always_inline)) {
    const int f = q % FC, w = q / FC;
    const bool isb = w >= 1 && w <= NB;
    const int blk = w == 0 ? 0 : (isb ? w - 1 : w - NB);
    const int r0 = (isb ? wn * NB : wm * MB) * 32 + blk * 32;   // first row of the block
    const char* unit = lds + (isb ? ub : ua);
    u32x4 v;
    if constexpr (AT || BT) {
      if (isb ? BT : AT)
        v = isb ? read_tr<NT>(unit, r0, s, lane) : read_tr<MT>(unit, r0, s, lane);
      else
        v = *reinterpret_cast<const u32x4*>(unit + (r0 + fr) * 128 + (((s * 2 + fg) * FC + f) ^ ((fr >> 1) & 7)) * 16);
    } else {
      v = *reinterpret_cast<const u32x4*>(unit + (r0 + fr) * 128 + (((s * 2 + fg) * FC + f) ^ ((fr >> 1) & 7)) * 16);
    }
    if (isb)
      F.b[blk < NB ? blk : 0][f] = v;
    else
      F.a[blk < MB ? blk : 0][f] = v;
  };
  auto scale = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int a = 0; a < MB; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[a][b][v] *= g.s;
  };

  // One step: its matrix instructions, and between them the next step's
  // fragment reads (in its first half) and loads [l0, l1) of the period's BPW,
  // the columns' first. Four waves that issue a stage's loads at once wait for
  // the address unit for half of the stage. The order is pinned: the compiler
  // keeps LDS reads and direct loads (which write LDS) in the order of the
  // source but not the matrix instructions between them.
  constexpr int RPM = (2 * ND + NM - 1) / NM;
  Frag F[2];
  // (B8: an eighth or sixteenth of the period's conversions, part t of STEPS, and
  // the rows' loads.)
  auto step = [&](Frag& cur, Frag& nxt, int ua, int ub, int s, int i, int ul, int um, int l0, int l1, int t, auto pair)
      __attribute__((always_inline)) {
    using TX = std::conditional_t<I8 && decltype(pair)::value, TP, T>;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int q = m * RPM; q < (m + 1) * RPM && q < ND; ++q)
        read(ua, ub, s, nxt, q);
      if constexpr (B8) {
#pragma unroll
        for (int l = 0; l < ABLK / STEPS; ++l)
          if (l * NM / (ABLK / STEPS) == m) issue_a8(i + P + 1, um, t * (ABLK / STEPS) + l);
#pragma unroll
        for (int e = m * PER_STEP / NM; e < (m + 1) * PER_STEP / NM; ++e) convert(ul, t * PER_STEP + e);
      } else {
#pragma unroll
        for (int l = l0; l < l1; ++l)
          if ((l - l0) * NM / (l1 - l0) == m) {
            if (l < BBLK)
              issue_b(i + P, ul, l);
            else
              issue_a(i + P + 1, um, l - BBLK);
          }
      }
      acc[m / NB][m % NB] = Op<TX>::run(cur.b[m % NB], cur.a[m / NB], acc[m / NB][m % NB]);   // (turned)
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Byte offset of the k-th unit after the current stage's rows.
  int u0 = 0;
  auto unit = [&](int k) __attribute__((always_inline)) {
    const int at = u0 + k * UNIT;
    return at >= RING ? at - RING : at;
  };
#pragma unroll
  for (int j = 0; j < (B8 ? 1 : P); ++j) {
#pragma unroll
    for (int b = 0; b < ABLK; ++b) {
      if constexpr (B8)
        issue_a8(st0, 0, b);
      else
        issue_a(st0 + j, 2 * j * UNIT, b);
    }
    if (!B8 && j + 1 < P) {
#pragma unroll
      for (int b = 0; b < BBLK; ++b) issue_b(st0 + j, (2 * j + 1) * UNIT, b);
    }
  }
  // (the columns of stage P - 1 and the rows of stage P: one period's loads, of
  // which the first step's part goes out here)
  constexpr int L1 = B8 ? ABLK / STEPS : BPW / STEPS;
  // Loads younger than the next stage's (B8: of the rows', after the last of which
  // come a period's rows and two loads for each of a lane's 16 bytes).
  constexpr int LATER = B8 ? ABLK + 2 * BBLK : (P - 1) * ABLK + (P - 2) * BBLK;
  if constexpr (B8) {
    // (In a period's order, so that the waits of the loop, which are those of its
    // first round too, leave as many loads in flight as its other rounds could.)
#pragma unroll
    for (int j = 0; j < BBLK; ++j) load_q(j);
#pragma unroll
    for (int t = 0; t <= STEPS; ++t) {
      const bool first = t < STEPS;
      if (t == 0 || t == STEPS) advance();
#pragma unroll
      for (int l = 0; l < L1; ++l)
        issue_a8(first ? st0 + 1 : st0 + 2, first ? 2 * UNIT : 4 * UNIT, (first ? t * L1 : 0) + l);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < PER_STEP; ++e)
        convert(first ? UNIT : 3 * UNIT, (first ? t * PER_STEP : 0) + e);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_vm_lgkm0<LATER + L1>();
  } else {
#pragma unroll
    for (int l = 0; l < L1; ++l) {
      if (l < BBLK)
        issue_b(st0 + P - 1, (2 * P - 1) * UNIT, l);
      else
        issue_a(st0 + P, 2 * P * UNIT, l - BBLK);
    }
    wait_vm_lgkm0<LATER + L1>();
  }
  barrier_keep_loads();
#pragma unroll
  for (int q = 0; q < ND; ++q) read(0, UNIT, 0, F[0], q);
  // Every matrix instruction stands in this one loop body: with the last
  // step's outside of it the compiler moved all accumulators between register
  // files around the loop.
  auto stage = [&](int i, auto pair) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s + 1 < STEPS; ++s)
      step(F[s & 1], F[(s + 1) & 1], unit(0), unit(1), s + 1, i - 1, unit(2 * P - 1), unit(2 * P),
           BPW * (s + 1) / STEPS, BPW * (s + 2) / STEPS, s + 1, pair);
    // This wave has read all of stage i, and its loads of stage i + 1 have
    // landed; younger ones stay in flight. Past the barrier the units of stage
    // i take the next period's loads.
    wait_vm_lgkm0<LATER>();
    barrier_keep_loads();
    if constexpr (B8) advance();
    step(F[1], F[0], unit(2), unit(3), 0, i, unit(0), unit(1), 0, L1, 0, pair);
    u0 = unit(2);
  };
  // Scales of the four columns that a lane holds in accumulators 4q to 4q + 3 of
  // a block, row lane % 32 of it (past the last column zeros).
  typedef float f32x4v __attribute__((ext_vector_type(4)));
  const __amdgpu_buffer_rsrc_t ws_rsrc = make_rsrc(g.w_scale, I8 ? (uint32_t)(g.N * 4) : 0u);
  auto w_scale4 = [&](int b, int q) __attribute__((always_inline)) {
    const int at = (int)(n0 + (wn * NB + b) * 32 + 8 * q + 4 * fg) * 4;
    return __builtin_bit_cast(f32x4v, __builtin_amdgcn_raw_buffer_load_b128(ws_rsrc, at, 0, 0));
  };
  int i = st0;
  if constexpr (I8) {
    const int mid = st1 < n1 ? st1 : n1;
    for (; i < mid; ++i) stage(i, Tag<false>{});
    // (Without a pair the epilogue converts the sums.)
    if constexpr (PAIR) {
      float rs[MB];
#pragma unroll
      for (int a = 0; a < MB; ++a) {
        const int64_t m = m0 + (wm * MB + a) * 32 + fr;
        rs[a] = g.pair_rows[m < g.M ? m : g.M - 1];
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4v ws = w_scale4(b, q);
#pragma unroll
          for (int a = 0; a < MB; ++a)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float sum = (float)__float_as_int(acc[a][b][4 * q + v]);
              acc[a][b][4 * q + v] = sum * rs[a] * ws[v] * g.inv_s;
            }
        }
      for (; i < st1; ++i) stage(i, Tag<true>{});
      scale();
    }
  } else {
    if constexpr (PAIR) {
      if (st0 < n2) {
        for (; i < n2; ++i) stage(i, Tag<true>{});
        scale();
      }
    }
    for (; i < st1; ++i) stage(i, Tag<false>{});
  }
  wait_vm_lgkm0<0>();   // (the loads past the depth too: the ring is reused)
  barrier_keep_loads();
  // Epilogue: each wave turns its accumulators, 32 rows at a time, into rows
  // of eight columns a lane through its own part of LDS, so that loads and
  // stores of the outputs are 16 bytes a lane along a row. (The operands were
  // given to the matrix instructions in turned order: a lane holds row lane %
  // 32 of a block and four consecutive columns in each four accumulators, so
  // that it writes 16 bytes at a time here too.)
  // The code is one real loop over pairs of passes: unrolled, its instructions
  // were fetched anew by every tile, which cost more than the loop. The
  // accumulators are named by constants in a chain of uniform branches, since
  // registers cannot be indexed. The residual's rows are loaded one pass ahead.
  float* ew = reinterpret_cast<float*>(lds) + wave * 32 * EPW;
  // 8-bit integers without a pair: the columns' scales, in LDS (there are no
  // registers for them beside the accumulators of the 256-row tile)
  float* wl = reinterpret_cast<float*>(lds) + NW * 32 * EPW + wave * NB * 32;
  if constexpr (I8 && !PAIR) {
#pragma unroll
    for (int i = lane; i < NB * 32; i += 64) {
      const int64_t c = n0 + wn * NB * 32 + i;
      wl[i] = g.w_scale[c < g.N ? c : g.N - 1];
    }
  }
  constexpr int IT = MB * PB / 2;
  const bool has_res = !B8 && g.ep.residual != nullptr && g.splits == 1;
  const int64_t m_first = m0 + wm * MB * 32 + lane / LPR;   // this lane's first row; the others RPP apart
  const int64_t rows_left = g.M - m_first;
  const int rl = nv <= 0 || rows_left <= 0 ? 0 : (int)(rows_left < MB * 32 ? rows_left : MB * 32);
  const int64_t pass = (int64_t)RPP * g.N;                  // elements from one pass to the next
  int64_t at = m_first * g.N + n;
  Raw8<O> next[2] = {};
  auto load_res = [&](int it, int64_t from) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if ((2 * it + i) * RPP < rl)
        next[i] = load_raw8<O>(static_cast<const O*>(g.ep.residual) + from + i * pass, nv);
  };
  if (has_res) load_res(0, at);
#pragma unroll 1
  for (int it = 0; it < IT; ++it, at += 2 * pass) {
    const Raw8<O> res[2] = {next[0], next[1]};
    if (has_res && it + 1 < IT) load_res(it + 1, at + 2 * pass);
    if (it % (PB / 2) == 0) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int c = 0; c < MB; ++c) {
        if (c != it / (PB / 2)) continue;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4v v = {acc[c][b][4 * q], acc[c][b][4 * q + 1], acc[c][b][4 * q + 2], acc[c][b][4 * q + 3]};
            if constexpr (I8 && !PAIR) v = __builtin_convertvector(__builtin_bit_cast(i32x4, v), f32x4v);
            *reinterpret_cast<f32x4v*>(ew + fr * EPW + b * 32 + 8 * q + 4 * fg) = v;
          }
      }
      __builtin_amdgcn_wave_barrier();
    }
    float v[16];
    int64_t m[2], off[2];
    bool ok[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = ((it % (PB / 2)) * 2 + i) * RPP + lane / LPR;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] = ew[row * EPW + col + e];
      if constexpr (I8 && !PAIR) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * i + e] *= wl[col + e];
      }
      m[i] = m_first + (2 * it + i) * RPP;
      off[i] = at + i * pass;
      ok[i] = (2 * it + i) * RPP < rl;
    }
    if (g.splits > 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v[8 * i + e];
        if (ok[i]) store8<float>(g.part + (int64_t)split * g.M * g.N + off[i], nv, o);
      }
    } else if constexpr (B8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = v[8 * i + e];
        if (g.ep.row_scale) {   // (uniform)
          const float rs = ok[i] ? g.ep.row_scale[m[i]] : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] *= rs;
        }
        if (ok[i]) store8<O>(static_cast<O*>(g.ep.y) + off[i], nv, o);
      }
    } else {
      epilogue_rows<O, 2>(g.ep, v, cs, bs, m, off, ok, nv, res);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows (a batch of single tokens): the product is one reading of w, and
// bound by memory. A workgroup owns 8 R columns (rows of w), its eight waves
// a contiguous eighth of the depth each, and w goes from memory straight into
// the operand registers of the 16x16 matrix instructions, two batches of
// BATCH steps in flight. The tokens are the other operand (8 TF of them), read
// from L2.
// A load instruction takes 128 bytes of each of eight rows (lane l: row l % 8,
// chunk l / 8). To the matrix instruction that is 16 rows of four chunks:
// rows i < 8 are w's rows with the even chunks and rows i >= 8 the same rows
// with the odd ones, and likewise for the tokens, so that of its 16 x 16 sums
// the two diagonal 8 x 8 blocks are wanted and are added at the end. It wastes
// half of the matrix cores, which idle here, for whole 128-byte lines:
// reading 8192 x 8192 bf16 takes 21 us so, 24 us in 64-byte pieces of 16 rows
// and 21 us in 1 KiB pieces; with 32 rows a workgroup (one workgroup a compute
// unit instead of two) each is 10 to 20% slower.
// The waves' sums are added in wave order through LDS, then the epilogue runs
// on one element a thread. Rows at any element address are read as they are;
// only the last partial step of the depth is read with bounds.
// A small product of more rows takes the same kernel, a workgroup for each
// 16 x 16 of the result: its eight waves share the depth that one wave of a
// 64-row tile walks alone.
// ---------------------------------------------------------------------------
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Op16;
template <>
struct Op16<bf16_t> {
  static __device__ __forceinline__ f32x4 run(const u32x4* a, const u32x4* b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[0]), __builtin_bit_cast(bf16x8, b[0]),
                                                   c, 0, 0, 0);
  }
};
template <>
struct Op16<f16_t> {
  static __device__ __forceinline__ f32x4 run(const u32x4* a, const u32x4* b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a[0]), __builtin_bit_cast(f16x8, b[0]), c,
                                                  0, 0, 0);
  }
};
template <>
struct Op16<float> {
  static __device__ __forceinline__ f32x4 run(const u32x4* a, const u32x4* b, f32x4 c) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[0][e]), __uint_as_float(b[0][e]), c, 0, 0, 0);
    return c;
  }
};
template <>
struct Op16<e4m3_t> {
  static __device__ __forceinline__ f32x4 run(const u32x4* a, const u32x4* b, f32x4 c) {
    struct P {
      u32x4 lo, hi;
    };
    const P pa{a[0], a[1]}, pb{b[0], b[1]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, pa),
                                                            __builtin_bit_cast(i32x8, pb), c, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
  }
};

template <>
struct Op16<int8x_t> {   // integer sums, as in Op
  static __device__ __forceinline__ f32x4 run(const u32x4* a, const u32x4* b, f32x4 c) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(
                                         __builtin_bit_cast(i32x4, a[0]), __builtin_bit_cast(i32x4, b[0]),
                                         __builtin_bit_cast(i32x4, c), 0, 0, 0));
  }
};

constexpr int kFewWaves = 8;   // waves of a workgroup, each with its share of the depth

template <typename T, int R, int TF, int BATCH>
struct FewFrag {
  static constexpr int CH = std::is_same<T, e4m3_t>::value ? 2 : 1;   // 16-byte chunks a lane feeds one instruction
  u32x4 w[BATCH][R][CH], x[BATCH][TF][CH];
};

// Bytes [at, at + 16) of a row of `len` bytes, zeros past its end.
__device__ __forceinline__ u32x4 load_bounded(const char* row, int64_t at, int64_t len) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (at + 16 <= len) return *reinterpret_cast<const u32x4_any*>(row + at);
  if (at < len) {
    uint8_t tmp[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) tmp[e] = at + e < len ? (uint8_t)row[at + e] : (uint8_t)0;
    __builtin_memcpy(&v, tmp, 16);
  }
  return v;
}

// acc += this wave's share of the depth of one operand pair.
template <typename T, int R, int TF, int BATCH>
__device__ __forceinline__ void few_rows_depth(const char* const (&wp)[R], const char* const (&xp)[TF], int64_t len,
                                               int part, int parts, int chunk, f32x4 (&acc)[R][TF]) {
  using F = FewFrag<T, R, TF, BATCH>;
  constexpr int CH = F::CH, SB = 128 * CH;   // bytes of a row that one step takes
  const int64_t full = len / SB;            // whole steps
  const int64_t s0 = full * part / parts, s1 = full * (part + 1) / parts;
  const int64_t base = chunk * 16;
  auto load = [&](F& f, int64_t s, int n) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (i >= n) continue;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int64_t at = (s + i) * SB + c * 128 + base;
#pragma unroll
        for (int r = 0; r < R; ++r)
          f.w[i][r][c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(wp[r] + at));
#pragma unroll
        for (int t = 0; t < TF; ++t) f.x[i][t][c] = *reinterpret_cast<const u32x4_any*>(xp[t] + at);
      }
    }
  };
  auto run = [&](const F& f, int n) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (i >= n) continue;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TF; ++t) acc[r][t] = Op16<T>::run(f.w[i][r], f.x[i][t], acc[r][t]);
    }
  };
  F a, b;
  int64_t s = s0;
  if (s + BATCH <= s1) {
    load(a, s, BATCH);
    s += BATCH;
    for (; s + 2 * BATCH <= s1; s += 2 * BATCH) {
      load(b, s, BATCH);
      run(a, BATCH);
      load(a, s + BATCH, BATCH);
      run(b, BATCH);
    }
    run(a, BATCH);
  }
  for (; s < s1; ++s) {
    load(a, s, 1);
    run(a, 1);
  }
  if (part == parts - 1 && full * SB < len) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t at = full * SB + c * 128 + base;
#pragma unroll
      for (int r = 0; r < R; ++r) a.w[0][r][c] = load_bounded(wp[r], at, len);
#pragma unroll
      for (int t = 0; t < TF; ++t) a.x[0][t][c] = load_bounded(xp[t], at, len);
    }
    run(a, 1);
  }
}

template <typename T, typename O, int R, int TF, int BATCH>
__global__ __launch_bounds__(kFewWaves * 64, TF <= 2 ? 2 : 1) void matmul_few_rows_kernel(GemmArgs g) {
  constexpr int ESZ = Op<T>::esz;
  constexpr bool I8 = std::is_same<T, int8x_t>::value;   // (sums first, then the pair; see the tile kernel)
  using TP = typename PairType<T, O>::type;
  constexpr int ESZ2 = Op<TP>::esz;
  __shared__ float red[kFewWaves * R * TF * 256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i8 = lane & 7, chunk = lane >> 3;
  const int row_block = blockIdx.x / g.n_nt, split = row_block / g.n_mt;
  const int64_t n0 = (int64_t)(blockIdx.x - row_block * g.n_nt) * (8 * R);
  const int64_t m0 = (int64_t)(row_block - split * g.n_mt) * (8 * TF);
  // Columns and tokens past the end read the last one's and are not stored.
  const char *wp[R], *xp[TF], *bp[R], *tp[TF];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t n = n0 + r * 8 + i8 < g.N ? n0 + r * 8 + i8 : g.N - 1;
    wp[r] = static_cast<const char*>(g.b) + n * g.ldb * ESZ;
    bp[r] = static_cast<const char*>(g.b2) + n * g.ldb2 * ESZ2;
  }
#pragma unroll
  for (int t = 0; t < TF; ++t) {
    const int64_t m = m0 + t * 8 + i8 < g.M ? m0 + t * 8 + i8 : g.M - 1;
    xp[t] = static_cast<const char*>(g.a) + m * g.lda * ESZ;
    tp[t] = static_cast<const char*>(g.a2) + m * g.lda2 * ESZ2;
  }
  f32x4 acc[R][TF];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TF; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int part = split * kFewWaves + wave, parts = g.splits * kFewWaves;
  if (!I8 && g.K2 > 0) {
    few_rows_depth<TP, R, TF, BATCH < 2 ? BATCH : 2>(bp, tp, g.K2 * ESZ2, part, parts, chunk, acc);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TF; ++t) acc[r][t] *= g.s;
  }
  few_rows_depth<T, R, TF, BATCH>(wp, xp, g.K * ESZ, part, parts, chunk, acc);
  if constexpr (I8) {
    // Sum (i, j) of a 16 x 16 block is value i % 4 of lane 16 (i / 4) + j: columns
    // 4 (lane / 16) + v mod 8 of the block's eight, and token lane % 8.
    const bool pair = g.K2 > 0;
    float rs[TF];
#pragma unroll
    for (int t = 0; t < TF; ++t) {
      const int64_t m = m0 + t * 8 + i8;
      rs[t] = pair ? g.pair_rows[m < g.M ? m : g.M - 1] : 1.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float ws[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t n = n0 + r * 8 + 4 * ((lane >> 4) & 1) + v;
        ws[v] = g.w_scale[n < g.N ? n : g.N - 1];
      }
#pragma unroll
      for (int t = 0; t < TF; ++t) {
        const i32x4 sum = __builtin_bit_cast(i32x4, acc[r][t]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[r][t][v] = (float)sum[v] * rs[t] * ws[v] * (pair ? g.inv_s : 1.f);
      }
    }
    if (pair) {
      few_rows_depth<TP, R, TF, BATCH < 2 ? BATCH : 2>(bp, tp, g.K2 * ESZ2, part, parts, chunk, acc);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TF; ++t) acc[r][t] *= g.s;
    }
  }
  // Sum (i, j) of a 16 x 16 block is value i % 4 of lane 16 (i / 4) + j.
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TF; ++t)
      *reinterpret_cast<f32x4*>(red + ((wave * R + r) * TF + t) * 256 + lane * 4) = acc[r][t];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * R * TF; i += kFewWaves * 64) {
    const int nl = i % (8 * R), ml = i / (8 * R);
    const int64_t n = n0 + nl, m = m0 + ml;
    if (m >= g.M || n >= g.N) continue;
    const int at = ((nl / 8) * TF + ml / 8) * 256 + (16 * ((nl % 8) / 4) + ml % 8) * 4 + nl % 4;
    constexpr int kOther = (16 * 2 + 8) * 4;   // from sum (i, j) to sum (i + 8, j + 8)
    float v = red[at] + red[at + kOther];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += red[w * R * TF * 256 + at] + red[w * R * TF * 256 + at + kOther];
    if (g.splits > 1) {
      g.part[((int64_t)split * g.M + m) * g.N + n] = v;
    } else {
      const float cs1 = g.ep.col_scale ? g.ep.col_scale[n] : 1.f, bs1 = g.ep.bias ? g.ep.bias[n] : 0.f;
      epilogue1<O>(g.ep, v, cs1, bs1, m, m * g.N + n);
    }
  }
}

// Adds the parts of the depth in increasing order and runs the epilogue.
template <typename O>
__global__ __launch_bounds__(256) void matmul_join_kernel(GemmArgs g) {
  const int64_t strips = (g.N + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= g.M * strips) return;
  const int64_t m = i / strips, n = (i - m * strips) * 8;
  const int nv = (int)(g.N - n < 8 ? g.N - n : 8);
  float v[8];
  load8<float>(g.part + m * g.N + n, nv, v);
  for (int x = 1; x < g.splits; ++x) {
    float p[8];
    load8<float>(g.part + ((int64_t)x * g.M + m) * g.N + n, nv, p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += p[e];
  }
  float cs[8], bs[8];
  column_terms(g.ep, n, nv, cs, bs);
  const int64_t off = m * g.N + n;
  Raw8<O> res[1] = {};
  if (g.ep.residual) res[0] = load_raw8<O>(static_cast<const O*>(g.ep.residual) + off, nv);
  const int64_t ms[1] = {m}, offs[1] = {off};
  const bool ok[1] = {true};
  epilogue_rows<O, 1>(g.ep, v, cs, bs, ms, offs, ok, nv, res);
}

// Copies of up to four operands [rows][kb bytes] (rows one after the other, at
// any alignment) to rows of lb bytes (a multiple of 16), zeros from kb on, in
// one launch. Job j's 16-byte chunks are numbers [first[j], first[j + 1]).
struct PackJobs {
  const char* src[4];
  char* dst[4];
  int64_t kb[4], lb[4], first[5];
  int n;
};

__global__ __launch_bounds__(256) void pack_rows_kernel(PackJobs p) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.first[p.n]) return;
  const char* src = p.src[0];
  char* dst = p.dst[0];
  int64_t kb = p.kb[0], lb = p.lb[0], base = 0;
#pragma unroll
  for (int j = 1; j < 4; ++j)
    if (j < p.n && i >= p.first[j]) src = p.src[j], dst = p.dst[j], kb = p.kb[j], lb = p.lb[j], base = p.first[j];
  i -= base;
  const int64_t cpr = lb / 16, r = i / cpr, c = (i - r * cpr) * 16;
  *reinterpret_cast<u32x4*>(dst + r * lb + c) = load_bounded(src + r * kb, c, kb);
}

template <typename T, typename O, int WM, int WN, int MB, int NB, int P, bool PAIR, bool AT = false, bool BT = false,
          bool B8 = false>
hipError_t launch_tile(GemmArgs g, hipStream_t st) {
  constexpr int MT = WM * MB * 32, NT = WN * NB * 32;
  g.n_mt = (int)((g.M + MT - 1) / MT);
  g.n_nt = (int)((g.N + NT - 1) / NT);
  auto k = matmul_tile_kernel<T, O, WM, WN, MB, NB, P, PAIR, AT, BT, B8>;
  constexpr int lds = (2 * P + 1) * (MT > NT ? MT : NT) * 128;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k, dim3((unsigned)((int64_t)g.n_mt * g.n_nt * g.splits)), dim3(WM * WN * 64), lds, st, g);
  return hipGetLastError();
}

template <typename O>
hipError_t launch_join(const GemmArgs& g, hipStream_t st) {
  const int64_t n = g.M * ((g.N + 7) / 8);
  hipLaunchKernelGGL((matmul_join_kernel<O>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, g);
  return hipGetLastError();
}

template <typename T, typename O, int R, int TF>
hipError_t launch_few_rows(GemmArgs g, hipStream_t st) {
  g.n_nt = (int)((g.N + 8 * R - 1) / (8 * R));
  g.n_mt = (int)((g.M + 8 * TF - 1) / (8 * TF));
  // (at most 128 registers, two workgroups a compute unit, where TF <= 2)
  constexpr int BATCH = (TF == 1 ? 4 : 2) / (std::is_same<T, e4m3_t>::value ? 2 : 1);
  hipLaunchKernelGGL((matmul_few_rows_kernel<T, O, R, TF, BATCH>), dim3((unsigned)((int64_t)g.n_nt * g.n_mt * g.splits)),
                     dim3(kFewWaves * 64), 0, st, g);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || g.splits == 1 ? e : launch_join<O>(g, st);
}

// Stages of KT elements of the whole depth and of each of g.splits parts.
void split_stages(GemmArgs& g, int KT, int KT2) {
  const int n2 = (int)((g.K2 + KT2 - 1) / KT2);
  g.stages = n2 + (int)((g.K + KT - 1) / KT);
  if (g.stages < 1) g.stages = 1;   // (no depth at all: one stage of zeros)
  // The low-rank stages and their scaling belong to the first part alone
  // (8-bit integers, whose pair comes last: each part scales what it has).
  const int per = (g.stages + g.splits - 1) / g.splits;
  g.stages_per_split = per > n2 || KT != KT2 ? per : n2;
  g.splits = (g.stages + g.stages_per_split - 1) / g.stages_per_split;
}

// Adds a copy of *src to the jobs and points *src at it.
[[maybe_unused]] void add_pack(PackJobs& p, const void** src, int64_t rows, int64_t kb, int64_t lb, char* dst) {
  const int j = p.n++;
  p.src[j] = static_cast<const char*>(*src), p.dst[j] = dst, p.kb[j] = kb, p.lb[j] = lb;
  p.first[j + 1] = p.first[j] + rows * (lb / 16);
  *src = dst;
}

[[maybe_unused]] hipError_t launch_pack(const PackJobs& p, hipStream_t st) {
  if (p.n == 0 || p.first[p.n] == 0) return hipSuccess;
  hipLaunchKernelGGL(pack_rows_kernel, dim3((unsigned)((p.first[p.n] + 255) / 256)), dim3(256), 0, st, p);
  return hipGetLastError();
}

}  // namespace

}  // namespace dora
