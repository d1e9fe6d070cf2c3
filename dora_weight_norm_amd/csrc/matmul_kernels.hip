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
#include "dora_device.h"
#include "dora_launch.h"
#include "dora_matmul.h"

namespace dora {

namespace {

typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct e4m3_t {
  uint8_t v;
};

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
template <typename T, typename O, int WM, int WN, int MB, int NB, int P, bool PAIR, bool AT, bool BT>
__global__ __launch_bounds__(WM* WN * 64, 1) void matmul_tile_kernel(GemmArgs g) {
  constexpr int ESZ = Op<T>::esz, FC = Op<T>::fc, E = 16 / ESZ, KT = 128 / ESZ;
  constexpr int NW = WM * WN, MT = WM * MB * 32, NT = WN * NB * 32;
  constexpr int UNIT = (MT > NT ? MT : NT) * 128;           // bytes of a ring unit
  constexpr int ABLK = MT / 8 / NW, BBLK = NT / 8 / NW;   // 1 KiB blocks per wave per stage
  constexpr int BPW = ABLK + BBLK;
  constexpr int STEPS = 8 / (2 * FC);
  constexpr int EPW = NB * 32 + 4;                         // floats of an epilogue row (padded: no bank conflicts)
  static_assert(MT % (8 * NW) == 0 && NT % (8 * NW) == 0, "a stage splits evenly over the waves");
  constexpr int RING = (2 * P + 1) * UNIT;
  static_assert(NW * 32 * EPW * 4 <= RING, "the epilogue fits the ring");
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
  const Stream sa2 = make_stream<ESZ, MT, NW, false>(g.a2, g.lda2, m0, g.M, lane, wave);
  const Stream sb2 = make_stream<ESZ, NT, NW, false>(g.b2, g.ldb2, n0, g.N, lane, wave);
  // Stages: the low-rank pair's first, then the main depth's; this workgroup's
  // part of them is [st0, st1).
  const int n2 = PAIR ? (int)((g.K2 + KT - 1) / KT) : 0;
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
      const bool pr = PAIR && i < n2;
      const int k0 = (pr ? i : i - n2) * 128;   // bytes of depth before the stage
      const int left = i < st1 ? (int)((pr ? g.K2 : g.K) * ESZ) - k0 : 0;
      const uint32_t at = pr ? pair.off + (uint32_t)b * pair.step : main.off + (uint32_t)b * main.step;
      const uint32_t off = chunk * 16 < left ? at : kOob;
      const __amdgpu_buffer_rsrc_t rs = pr ? pair.rsrc : main.rsrc;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, off, k0, 0, 0);
    }
  };
  auto issue_a = [&](int i, int unit, int b) __attribute__((always_inline)) { issue(sa, sa2, i, unit, b, Tag<AT>{}); };
  auto issue_b = [&](int i, int unit, int b) __attribute__((always_inline)) { issue(sb, sb2, i, unit, b, Tag<BT>{}); };

  // The epilogue's columns of this lane: their scales and biases are asked for
  // here, a whole depth before they are needed.
  constexpr int LPR = NB * 4, RPP = 64 / LPR, PB = 32 / RPP;   // lanes a row, rows a pass, passes a block
  const int col = (lane % LPR) * 8;
  const int64_t n = n0 + wn * NB * 32 + col;
  const int nv = (int)(g.N - n < 8 ? g.N - n : 8);
  float cs[8], bs[8];
  column_terms(g.ep, n, nv, cs, bs);

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
  auto step = [&](Frag& cur, Frag& nxt, int ua, int ub, int s, int i, int ul, int um, int l0, int l1)
      __attribute__((always_inline)) {
#pragma unroll
    for (int m = 0; m < NM; ++m) {
#pragma unroll
      for (int q = m * RPM; q < (m + 1) * RPM && q < ND; ++q)
        read(ua, ub, s, nxt, q);
#pragma unroll
      for (int l = l0; l < l1; ++l)
        if ((l - l0) * NM / (l1 - l0) == m) {
          if (l < BBLK)
            issue_b(i + P, ul, l);
          else
            issue_a(i + P + 1, um, l - BBLK);
        }
      acc[m / NB][m % NB] = Op<T>::run(cur.b[m % NB], cur.a[m / NB], acc[m / NB][m % NB]);   // (turned)
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
  for (int j = 0; j < P; ++j) {
#pragma unroll
    for (int b = 0; b < ABLK; ++b) issue_a(st0 + j, 2 * j * UNIT, b);
    if (j + 1 < P) {
#pragma unroll
      for (int b = 0; b < BBLK; ++b) issue_b(st0 + j, (2 * j + 1) * UNIT, b);
    }
  }
  // (the columns of stage P - 1 and the rows of stage P: one period's loads, of
  // which the first step's part goes out here)
  constexpr int L1 = BPW / STEPS;
  constexpr int LATER = (P - 1) * ABLK + (P - 2) * BBLK;   // loads younger than the next stage's
#pragma unroll
  for (int l = 0; l < L1; ++l) {
    if (l < BBLK)
      issue_b(st0 + P - 1, (2 * P - 1) * UNIT, l);
    else
      issue_a(st0 + P, 2 * P * UNIT, l - BBLK);
  }
  wait_vm_lgkm0<LATER + L1>();
  barrier_keep_loads();
#pragma unroll
  for (int q = 0; q < ND; ++q) read(0, UNIT, 0, F[0], q);
  // Every matrix instruction stands in this one loop body: with the last
  // step's outside of it the compiler moved all accumulators between register
  // files around the loop.
  auto stage = [&](int i) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s + 1 < STEPS; ++s)
      step(F[s & 1], F[(s + 1) & 1], unit(0), unit(1), s + 1, i - 1, unit(2 * P - 1), unit(2 * P),
           BPW * (s + 1) / STEPS, BPW * (s + 2) / STEPS);
    // This wave has read all of stage i, and its loads of stage i + 1 have
    // landed; younger ones stay in flight. Past the barrier the units of stage
    // i take the next period's loads.
    wait_vm_lgkm0<LATER>();
    barrier_keep_loads();
    step(F[1], F[0], unit(2), unit(3), 0, i, unit(0), unit(1), 0, L1);
    u0 = unit(2);
  };
  int i = st0;
  if constexpr (PAIR) {
    if (st0 < n2) {
      for (; i < n2; ++i) stage(i);
      scale();
    }
  }
  for (; i < st1; ++i) stage(i);
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
  constexpr int IT = MB * PB / 2;
  const bool has_res = g.ep.residual != nullptr && g.splits == 1;
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
            typedef float f32x4v __attribute__((ext_vector_type(4)));
            const f32x4v v = {acc[c][b][4 * q], acc[c][b][4 * q + 1], acc[c][b][4 * q + 2], acc[c][b][4 * q + 3]};
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

constexpr int kFewWaves = 8;   // waves of a workgroup, each with its share of the depth

template <typename T, int R, int TF, int BATCH>
struct FewFrag {
  static constexpr int CH = sizeof(T) == 1 ? 2 : 1;   // 16-byte chunks a lane feeds one instruction
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
    bp[r] = static_cast<const char*>(g.b2) + n * g.ldb2 * ESZ;
  }
#pragma unroll
  for (int t = 0; t < TF; ++t) {
    const int64_t m = m0 + t * 8 + i8 < g.M ? m0 + t * 8 + i8 : g.M - 1;
    xp[t] = static_cast<const char*>(g.a) + m * g.lda * ESZ;
    tp[t] = static_cast<const char*>(g.a2) + m * g.lda2 * ESZ;
  }
  f32x4 acc[R][TF];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TF; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int part = split * kFewWaves + wave, parts = g.splits * kFewWaves;
  if (g.K2 > 0) {
    few_rows_depth<T, R, TF, BATCH < 2 ? BATCH : 2>(bp, tp, g.K2 * ESZ, part, parts, chunk, acc);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TF; ++t) acc[r][t] *= g.s;
  }
  few_rows_depth<T, R, TF, BATCH>(wp, xp, g.K * ESZ, part, parts, chunk, acc);
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

// dst[c][r] = src[r][c] for src [rows][cols] at row stride lds_; dst rows of
// stride ld >= rows, zeros from `rows` on. 64 x 64 tiles through LDS.
template <typename U>
__global__ __launch_bounds__(256) void transpose_kernel(const U* src, int64_t rows, int64_t cols, int64_t lsrc,
                                                        int64_t ld, U* dst) {
  __shared__ U tile[64][65];
  const int64_t nr = (ld + 63) / 64;   // row tiles (of the destination's stride, so that its padding is written)
  const int64_t r0 = blockIdx.x % nr * 64, c0 = blockIdx.x / nr * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + i * 4 + ty, c = c0 + tx;
    tile[i * 4 + ty][tx] = (r < rows && c < cols) ? src[r * lsrc + c] : U(0);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t c = c0 + i * 4 + ty, r = r0 + tx;
    if (c < cols && r < ld) dst[c * ld + r] = tile[tx][i * 4 + ty];
  }
}

// Element-wise part of the backward: z from u, dz = dy act'(z), du = row_scale
// col_scale dz (rounded to the storage type: it is the operand of both
// products, which the matrix cores take in 16 bits), and this row block's sums
// of dz and dz u over its rows, in increasing order (u holds the row scale).
template <typename T>
__global__ __launch_bounds__(256) void matmul_bwd_kernel(const T* dy, const T* u, const float* row_scale,
                                                         const float* col_scale, const float* bias, int act, int64_t M,
                                                         int64_t N, T* du, int64_t ldu, T* du2, float* sums) {
  __shared__ float lanes[16][256];
  const int64_t strip = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t n = strip * 8;
  const int ly = threadIdx.y, nl = blockDim.y;
  const int nv = (int)(N - n < 8 ? (N - n < 0 ? 0 : N - n) : 8);
  float cs[8], bs[8], sb[8], sc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e] = (col_scale && e < nv) ? col_scale[n + e] : 1.f;
    bs[e] = (bias && e < nv) ? bias[n + e] : 0.f;
    sb[e] = sc[e] = 0.f;
  }
  // Four rows' loads are in flight at a time.
  constexpr int U = 4;
  const int64_t step = (int64_t)gridDim.y * nl;
  for (int64_t m0 = (int64_t)blockIdx.y * nl + ly; nv > 0 && m0 < M; m0 += U * step) {
    Raw8<T> ry[U], ru[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t m = m0 + i * step;
      if (m < M) {
        // (du, which the products read next, is to stay in the caches)
        ry[i] = load_raw8<T, true>(dy + m * N + n, nv);
        ru[i] = load_raw8<T, true>(u + m * N + n, nv);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t m = m0 + i * step;
      if (m >= M) continue;
      const float rs = row_scale ? row_scale[m] : 1.f;
      float y[8], v[8], o[8];
      unpack8<T>(ry[i], y);
      unpack8<T>(ru[i], v);
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
      if (nv < 8 && ldu > N) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (e >= nv) o[e] = 0.f;
        store8<T>(du + m * ldu + n, (int)(ldu - n < 8 ? ldu - n : 8), o);
      } else {
        store8<T>(du + m * ldu + n, nv, o);
      }
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
int stage_depth(int dtype) { return dtype == 1 ? 32 : (dtype == 3 ? 128 : 64); }
int elem_size(int dtype) { return dtype == 1 ? 4 : (dtype == 3 ? 1 : 2); }
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

template <typename T, typename O, int WM, int WN, int MB, int NB, int P, bool PAIR, bool AT = false, bool BT = false>
hipError_t launch_tile(GemmArgs g, hipStream_t st) {
  constexpr int MT = WM * MB * 32, NT = WN * NB * 32;
  g.n_mt = (int)((g.M + MT - 1) / MT);
  g.n_nt = (int)((g.N + NT - 1) / NT);
  auto k = matmul_tile_kernel<T, O, WM, WN, MB, NB, P, PAIR, AT, BT>;
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
  constexpr int BATCH = (TF == 1 ? 4 : 2) / (Op<T>::esz == 1 ? 2 : 1);
  hipLaunchKernelGGL((matmul_few_rows_kernel<T, O, R, TF, BATCH>), dim3((unsigned)((int64_t)g.n_nt * g.n_mt * g.splits)),
                     dim3(kFewWaves * 64), 0, st, g);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || g.splits == 1 ? e : launch_join<O>(g, st);
}

// Stages of KT elements of the whole depth and of each of g.splits parts.
void split_stages(GemmArgs& g, int KT) {
  const int n2 = (int)((g.K2 + KT - 1) / KT);
  g.stages = n2 + (int)((g.K + KT - 1) / KT);
  if (g.stages < 1) g.stages = 1;   // (no depth at all: one stage of zeros)
  // The low-rank stages and their scaling belong to the first part alone.
  const int per = (g.stages + g.splits - 1) / g.splits;
  g.stages_per_split = per > n2 ? per : n2;
  g.splits = (g.stages + g.stages_per_split - 1) / g.stages_per_split;
}

// The backward's products on operands as they lie (16-bit types): `b` stored
// [k][row], and with AT `a` too.
template <typename T, bool AT>
hipError_t launch_gemm_tr(GemmArgs g, int cfg, hipStream_t st) {
  split_stages(g, 64);
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
  split_stages(g, 128 / Op<T>::esz);
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

// Adds a copy of *src to the jobs and points *src at it.
void add_pack(PackJobs& p, const void** src, int64_t rows, int64_t kb, int64_t lb, char* dst) {
  const int j = p.n++;
  p.src[j] = static_cast<const char*>(*src), p.dst[j] = dst, p.kb[j] = kb, p.lb[j] = lb;
  p.first[j + 1] = p.first[j] + rows * (lb / 16);
  *src = dst;
}

hipError_t launch_pack(const PackJobs& p, hipStream_t st) {
  if (p.n == 0 || p.first[p.n] == 0) return hipSuccess;
  hipLaunchKernelGGL(pack_rows_kernel, dim3((unsigned)((p.first[p.n] + 255) / 256)), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t transpose(const void* src, int64_t rows, int64_t cols, int64_t lsrc, int64_t ld, int esz, void* dst,
                     hipStream_t st) {
  const dim3 grid((unsigned)((ld + 63) / 64 * ((cols + 63) / 64)));
  if (esz == 2)
    hipLaunchKernelGGL((transpose_kernel<uint16_t>), grid, dim3(256), 0, st, static_cast<const uint16_t*>(src), rows,
                       cols, lsrc, ld, static_cast<uint16_t*>(dst));
  else
    hipLaunchKernelGGL((transpose_kernel<uint32_t>), grid, dim3(256), 0, st, static_cast<const uint32_t*>(src), rows,
                       cols, lsrc, ld, static_cast<uint32_t*>(dst));
  return hipGetLastError();
}

}  // namespace

MatmulPlan plan_matmul(int64_t M, int64_t N, int64_t K, int64_t r, int dtype, int al) {
  MatmulPlan p{};
  const int esz = elem_size(dtype), epc = 16 / esz, KT = stage_depth(dtype);
  size_t off = 0;
  choose_tile(M, N, up(K, KT) / KT, dtype, K % epc == 0 ? kFewOnGrid : kFewOffGrid, &p.cfg, &p.splits);
  auto operand = [&](int64_t rows, int64_t depth, int bit, bool* pack, int64_t* ld, size_t* at) {
    // (the few-rows kernel reads rows at any element address)
    *pack = p.cfg < kFew8 && depth > 0 && (depth % epc != 0 || !(al & bit));
    *ld = *pack ? up(depth, epc) : depth;
    *at = off;
    if (*pack) off = up256(off + (size_t)(rows * *ld) * esz);
  };
  operand(M, K, 1, &p.pack_x, &p.ldx, &p.off_x);
  operand(N, K, 2, &p.pack_w, &p.ldw, &p.off_w);
  operand(M, r, 4, &p.pack_t, &p.ldt, &p.off_t);
  operand(N, r, 8, &p.pack_b, &p.ldb, &p.off_b);
  p.off_part = off;
  if (p.splits > 1) off = up256(off + (size_t)(p.splits * M * N) * 4);
  p.ws_bytes = off;
  return p;
}

hipError_t launch_matmul(const MatmulPlan& p, const void* x, const void* w, int dtype, int64_t M, int64_t N,
                         int64_t K, const void* t, const void* b, int64_t r, float s, const Epilogue& ep,
                         int out_dtype, char* ws, hipStream_t st) {
  const int esz = elem_size(dtype);
  PackJobs jobs{};
  if (p.pack_x) add_pack(jobs, &x, M, K * esz, p.ldx * esz, ws + p.off_x);
  if (p.pack_w) add_pack(jobs, &w, N, K * esz, p.ldw * esz, ws + p.off_w);
  if (p.pack_t) add_pack(jobs, &t, M, r * esz, p.ldt * esz, ws + p.off_t);
  if (p.pack_b) add_pack(jobs, &b, N, r * esz, p.ldb * esz, ws + p.off_b);
  const hipError_t e = launch_pack(jobs, st);
  if (e != hipSuccess) return e;
  GemmArgs g{};
  g.a = x, g.b = w, g.lda = p.ldx, g.ldb = p.ldw, g.K = K;
  g.a2 = r > 0 ? t : nullptr, g.b2 = r > 0 ? b : nullptr, g.lda2 = p.ldt, g.ldb2 = p.ldb, g.K2 = r;
  g.s = s, g.M = M, g.N = N, g.splits = p.splits;
  g.part = reinterpret_cast<float*>(ws + p.off_part);
  g.ep = ep;
  return gemm(g, dtype, out_dtype, p.cfg, st);
}

MatmulBackwardPlan plan_matmul_backward(int64_t M, int64_t N, int64_t K, int dtype, bool need_dx, bool need_dw,
                                        bool need_sums, bool du_direct, bool aligned_xw) {
  MatmulBackwardPlan p{};
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
  p.off_du = take(p.du_direct ? 0 : (size_t)(M * p.ldn) * esz);
  p.off_sum = take(need_sums ? (size_t)(p.rows * 2 * N) * 4 : 0);
  // 16-bit products read du, w and x as they lie, copied to whole chunks where
  // their rows are none; fp32 ones (whose elements no transposing read takes)
  // read transposed copies.
  p.direct = dtype != 1;
  p.ldk = up(K, epc);
  p.copy = p.direct && (!aligned_xw || K % epc != 0);
  p.off_wt = take(!need_dx ? 0 : (p.copy ? (size_t)(N * p.ldk) * esz : (p.direct ? 0 : (size_t)(K * p.ldn) * esz)));
  p.off_dut = take(need_dw && !p.direct ? (size_t)(N * p.ldm) * esz : 0);
  p.off_xt = take(!need_dw ? 0 : (p.copy ? (size_t)(M * p.ldk) * esz : (p.direct ? 0 : (size_t)(K * p.ldm) * esz)));
  size_t part = 0;
  if (need_dx) {
    choose_tile(M, K, up(N, KT) / KT, dtype, p.direct ? 0 : kFewOnGrid, &p.cfg_dx, &p.splits_dx);
    if (p.splits_dx > 1) part = (size_t)(p.splits_dx * M * K) * 4;
  }
  if (need_dw) {
    choose_tile(N, K, up(M, KT) / KT, dtype, p.direct ? 0 : kFewOnGrid, &p.cfg_dw, &p.splits_dw);
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
                                  float* dbias, float* dcol, char* ws, hipStream_t st) {
  const int esz = elem_size(dtype);
  hipError_t e = hipSuccess;
  // The element-wise pass writes du into the caller's array where that can be
  // the products' operand, else at a padded row stride into the workspace
  // (and into the caller's array beside it).
  char* d = p.du_direct ? static_cast<char*>(du) : ws + p.off_du;
  void* du2 = p.du_direct ? nullptr : du;
  // (without rows the workspace may be null: whether sums are wanted is not read off their address)
  const bool want_sums = dbias || dcol;
  float* sums = want_sums ? reinterpret_cast<float*>(ws + p.off_sum) : nullptr;
  if (M > 0 && N > 0) {
    const int64_t strips = (N + 7) / 8;
    int64_t tx = up(strips, 64);
    if (tx > 256) tx = 256;
    const dim3 block((unsigned)tx, (unsigned)(256 / tx));
    const dim3 grid((unsigned)((strips + tx - 1) / tx), (unsigned)p.rows);
#define DORA_BWD(T)                                                                                             \
  hipLaunchKernelGGL((matmul_bwd_kernel<T>), grid, block, 0, st, static_cast<const T*>(dy),                     \
                     static_cast<const T*>(u), row_scale, col_scale, bias, act, M, N, reinterpret_cast<T*>(d),  \
                     p.ldn, static_cast<T*>(du2), sums)
    switch (dtype) {
      case 0: DORA_BWD(bf16_t); break;
      case 2: DORA_BWD(f16_t); break;
      default: DORA_BWD(float); break;
    }
#undef DORA_BWD
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (want_sums && N > 0) {
    e = launch_column_sum(sums, M > 0 ? (int)p.rows : 0, 2 * N, dbias, N, dcol, st);
    if (e != hipSuccess) return e;
  }
  GemmArgs g{};
  g.part = reinterpret_cast<float*>(ws + p.off_part);
  if (p.direct) {
    if (p.copy) {
      PackJobs jobs{};
      if (dx) add_pack(jobs, &w, N, K * esz, p.ldk * esz, ws + p.off_wt);
      if (dw) add_pack(jobs, &x, M, K * esz, p.ldk * esz, ws + p.off_xt);
      e = launch_pack(jobs, st);
      if (e != hipSuccess) return e;
    }
    const int64_t ldu = p.du_direct ? N : p.ldn, ldk = p.copy ? p.ldk : K;
    // dx: du along the depth, w across it; dw: both across it.
    if (dx && M > 0 && K > 0) {
      g.a = d, g.b = w, g.lda = ldu, g.ldb = ldk, g.K = N, g.M = M, g.N = K, g.splits = p.splits_dx;
      g.ep.y = dx;
      e = dtype == 0 ? launch_gemm_tr<bf16_t, false>(g, p.cfg_dx, st) : launch_gemm_tr<f16_t, false>(g, p.cfg_dx, st);
      if (e != hipSuccess) return e;
    }
    if (dw && N > 0 && K > 0) {
      g.a = d, g.b = x, g.lda = ldu, g.ldb = ldk, g.K = M, g.M = N, g.N = K, g.splits = p.splits_dw;
      g.ep.y = dw;
      e = dtype == 0 ? launch_gemm_tr<bf16_t, true>(g, p.cfg_dw, st) : launch_gemm_tr<f16_t, true>(g, p.cfg_dw, st);
    }
    return e;
  }
  if (dx && M > 0 && K > 0) {
    if (N > 0) e = transpose(w, N, K, K, p.ldn, esz, ws + p.off_wt, st);
    if (e != hipSuccess) return e;
    g.a = d, g.b = ws + p.off_wt, g.lda = p.ldn, g.ldb = p.ldn, g.K = N, g.M = M, g.N = K, g.splits = p.splits_dx;
    g.ep.y = dx;
    e = gemm(g, dtype, dtype, p.cfg_dx, st);
    if (e != hipSuccess) return e;
  }
  if (dw && N > 0 && K > 0) {
    if (M > 0) {
      e = transpose(d, M, N, p.ldn, p.ldm, esz, ws + p.off_dut, st);
      if (e != hipSuccess) return e;
      e = transpose(x, M, K, K, p.ldm, esz, ws + p.off_xt, st);
      if (e != hipSuccess) return e;
    }
    g.a = ws + p.off_dut, g.b = ws + p.off_xt, g.lda = p.ldm, g.ldb = p.ldm, g.K = M, g.M = N, g.N = K;
    g.splits = p.splits_dw;
    g.ep.y = dw;
    e = gemm(g, dtype, dtype, p.cfg_dw, st);
  }
  return e;
}

}  // namespace dora
