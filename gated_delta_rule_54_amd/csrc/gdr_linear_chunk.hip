// Linear attention with a decay for each head on the matrix cores: chunks of
// C tokens.  With A_i the running sum of the log decay up to row i of a chunk
// (in 64 bits: differences of far sums must keep the near ones' precision),
// a chain (gdr_linear.h) over one chunk is
//     P = (X Y^T) o e^{A_i - A_j}   (j <= i),
//     O = e^{A_i} X H + P Z,
//     H <- e^{A_C} H + Y^T (e^{A_C - A_j} Z).
// A chain backward in time is the same with the rows taken last to first and
// A_i the sum over the rows before i (the tokens after it).
//
// One workgroup walks a segment of a sequence for one value head and a slice
// of 64 columns with eight waves.  Waves 4 .. 7 carry the state: each keeps 16
// columns of H in accumulators for the whole walk and leaves H in LDS, as
// operands, for the chunk that comes.  Waves 0 .. 3 form the output from it.
// So the two products that depend on each other along the sequence (H, and
// what is read from it) run side by side, on one SIMD an output wave beside a
// state wave.  Accumulators are operands without a move: H's tile t takes rows
// 32 (t / 2) + 8 g + 4 (t % 2) + e (lane group g, element e), which is the
// order of X's operands.  O is formed transposed, a lane storing 4 consecutive
// columns of one token.  Output waves share the work by rows (out_by_rows)
// where H is one or two operands, by columns (out_by_columns) where it is three.
//
// Bound: waits.  4 x 4096 tokens, 16 key and 32 value heads of 128, bf16:
// forward 172-197 us (its bytes alone 67 us), VJP 673-870 us (bytes 110 us), of
// which dg 19-23: the least over the same buffers, the most within a layer.  That
// is 2.7-3.1 us a chunk of 64 tokens and 64 columns forward, 3.5-4.8 in the VJP.
// Counters there: the matrix cores are busy 25 % of the forward's time (22-25 %
// of the VJP's), LDS 47 % (37-44 %), over a third of that for bank conflicts.  Of
// a wave's time 42 % is waiting for LDS, memory or a barrier, 22 % for its turn to
// issue, 36 % issuing: two waves on a SIMD are too few to fill any of the units.
// Measured and set aside: 32 columns a wave (spills), chunks of 32 with two
// workgroups a compute unit, the state's update after the output in the same waves
// (262 us forward against 186, with one operand), output by columns also where H
// is two operands (175 against 174 us; 17 ragged sequences 224 against 221).
//
// Precision.  bf16 inputs are matrix-core operands as they are.  What is
// computed on the way (P, H, the decayed Z) is fp32: where a result is
// returned in fp32, or a sum over all tokens is (the state; the terms of the
// decay's gradient), it enters the product as a sum of three bf16 values (24
// bits); otherwise, for an output that is rounded to bf16 itself, as two (16
// bits: the error before the output's rounding is 2^-8 of that rounding's).  One
// (8 bits) is as coarse as the output: the 2-norm error is then 2.1e-3 where the
// rounding alone gives 1.7e-3, and the forward above takes 150 us instead of 174,
// the VJP 655 instead of 683.  fp32 inputs use fp32 operands.

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gdr_device.h"
#include "gdr_linear.h"

namespace gdr {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

__device__ __forceinline__ double dpp_add(double x, int lo, int hi) {
  return x + __builtin_bit_cast(double, (static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) |
                                            static_cast<uint32_t>(lo));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_step(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return dpp_add(x, __builtin_amdgcn_update_dpp(0, static_cast<int>(u), CTRL, ROWS, 0xf, false),
                 __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), CTRL, ROWS, 0xf, false));
}
// Inclusive prefix sum over the wave's lanes (the steps of wave_prefix_sum).
__device__ __forceinline__ double prefix64(double x) {
  x = dpp_step<0x111, 0xf>(x);
  x = dpp_step<0x112, 0xf>(x);
  x = dpp_step<0x114, 0xf>(x);
  x = dpp_step<0x118, 0xf>(x);
  x = dpp_step<0x142, 0xa>(x);
  return dpp_step<0x143, 0xc>(x);
}

// The value of the first lane of each row of 16, of the wave's last lane.
__device__ __forceinline__ double row_first(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(u), 0x150, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(u >> 32), 0x150, 0xf, 0xf, false);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double last_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(u), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(u >> 32), 63);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// log2 of a token's decay factor.  A factor below 2^-185 is zero in every
// product; the bound keeps -Inf out of the differences of sums.
__device__ __forceinline__ double log2_decay(float g) {
  return (g < -128.f ? -128.0 : static_cast<double>(g)) * 1.4426950408889634;
}

// Matrix-core operands: lane group g holds steps 8g .. 8g + 7 of a 32-step
// block of the summed index.  C chunk rows; PAD elements between LDS rows; PER
// elements of a 16-byte unit; FULL operands hold an fp32 value, NARROW one that
// is enough for a result in bf16.
template <int CC>
struct OpB {
  using E = uint16_t;
  static constexpr int C = CC, PAD = 8, PER = 8, FULL = 3, NARROW = 2;
  typedef bf16x8 F;
  static __device__ __forceinline__ F run(const E* p) { return *reinterpret_cast<const F*>(p); }
  // Rows k0 + 8g .. +7 of column n0 + step (p / 4) + p % 4, p = lane % 16, of
  // a row-major tile: one transposing read hands a group of 16 lanes 4 rows of
  // four runs of 4 columns.
  static __device__ __forceinline__ F col(const E* M, int ld, int k0, int n0, int step) {
    const int p = lane_id() & 15, g = lane_id() >> 4;
    const E* at = M + (k0 + 8 * g + (p >> 2)) * ld + n0 + step * (p & 3);
    const bf16x4 a = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
    const bf16x4 b = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * ld)));
    return F{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  // columns j .. j + 7 of row i of P (place as p_at)
  static __device__ __forceinline__ F prun(const E* P, int i, int j) {
    return run(P + i * C + ((j / 8) ^ (i & (C / 8 - 1))) * 8);
  }
  // Rows k0 + 4g .. +3 and k0 + 16 + 4g .. +3 of column n0 + lane % 16.
  static __device__ __forceinline__ F pair(const E* M, int ld, int k0, int n0) {
    const int p = lane_id() & 15, g = lane_id() >> 4;
    const E* at = M + (k0 + 4 * g + (p >> 2)) * ld + n0 + 4 * (p & 3);
    const bf16x4 a = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
    const bf16x4 b = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * ld)));
    return F{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ f32x4 mma(F a, F b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ void widen(float (&x)[8], F f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = __builtin_bit_cast(u32x4, f)[i];
      x[2 * i] = __uint_as_float(w << 16), x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
  }
  // Two values as NS bf16 pairs: each pair rounds what the ones before leave.
  template <int NS>
  static __device__ __forceinline__ void split2(uint32_t (&w)[NS], float a, float b) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      typedef float f2 __attribute__((ext_vector_type(2)));
      w[s] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
      a -= __uint_as_float(w[s] << 16);
      b -= __uint_as_float(w[s] & 0xffff0000u);
    }
  }
  // x as a sum of NS operands
  template <int NS>
  static __device__ __forceinline__ void split(F (&f)[NS], const float (&x)[8]) {
    uint32_t w[4][NS];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<NS>(w[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int s = 0; s < NS; ++s) f[s] = __builtin_bit_cast(F, (u32x4{w[0][s], w[1][s], w[2][s], w[3][s]}));
  }
  // x[0..3] into NS tiles, `step` elements apart, at p
  template <int NS>
  static __device__ __forceinline__ void put4(E* p, int step, f32x4 x) {
    uint32_t w[2][NS];
    split2<NS>(w[0], x[0], x[1]);
    split2<NS>(w[1], x[2], x[3]);
#pragma unroll
    for (int s = 0; s < NS; ++s) *reinterpret_cast<u32x2*>(p + s * step) = u32x2{w[0][s], w[1][s]};
  }
};

struct OpF {
  using E = float;
  static constexpr int C = 32, PAD = 4, PER = 4, FULL = 1, NARROW = 1;
  struct F { float v[8]; };
  static __device__ __forceinline__ F run(const E* p) {
    F f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = p[i];
    return f;
  }
  static __device__ __forceinline__ F col(const E* M, int ld, int k0, int n0, int step) {
    const int p = lane_id() & 15;
    const E* at = M + (k0 + 8 * (lane_id() >> 4)) * ld + n0 + step * (p >> 2) + (p & 3);
    F f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = at[i * ld];
    return f;
  }
  static __device__ __forceinline__ F pair(const E* M, int ld, int k0, int n0) {
    const E* at = M + (k0 + 4 * (lane_id() >> 4)) * ld + n0 + (lane_id() & 15);
    F f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = at[i * ld], f.v[4 + i] = at[(16 + i) * ld];
    return f;
  }
  static __device__ __forceinline__ f32x4 mma(const F& a, const F& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ void widen(float (&x)[8], const F& f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = f.v[i];
  }
  template <int NS>
  static __device__ __forceinline__ void split(F (&f)[NS], const float (&x)[8]) {
    static_assert(NS == 1, "fp32 operands are exact");
#pragma unroll
    for (int i = 0; i < 8; ++i) f[0].v[i] = x[i];
  }
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, uint32_t nbytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(nbytes), 0x00020000);
}

// A chunk's rows of one tensor as a buffer that ends with them: row i of the
// chunk lies i rows from its start, or, backward in time, n - 1 - i.  Reads
// outside give zeros, writes are dropped: rows at or past n lie beyond the end
// either way (backward as negative offsets, which wrap around), and kNone does.
constexpr uint32_t kNone = 0xf0000000u;
struct Rows {
  const char* top;  // row 0 of the chunk
  uint32_t rowb;    // bytes between tokens; a chunk's rows span less than 2^30 bytes
  uint32_t width;   // bytes of a row that may be touched
  bool rev;
  __device__ __forceinline__ rsrc_t chunk(int n) const {
    return make_rsrc(rev ? top - (n - 1) * rowb : top, (n - 1) * rowb + width);
  }
  __device__ __forceinline__ void next(int C) {
    const int64_t d = static_cast<int64_t>(C * rowb);
    top += rev ? -d : d;
  }
  // Offset of row i, from the chunk's n = C form.
  __device__ __forceinline__ uint32_t row(int i, int C) const { return (rev ? C - 1 - i : i) * rowb; }
  __device__ __forceinline__ uint32_t shift(int n, int C) const { return rev ? (C - n) * rowb : 0; }
  __device__ __forceinline__ uint32_t step(int k) const { return rev ? -(k * rowb) : k * rowb; }
};

// Rows of a chunk on their way from memory to LDS by NTH threads: 16-byte unit
// e of the [C][W] tile is loaded by thread e % NTH in round e / NTH.
template <typename OP, int W, int NTH>
struct Stage {
  static constexpr int UPR = W / OP::PER, UNITS = OP::C * UPR, N = (UNITS + NTH - 1) / NTH, STEP = NTH / UPR;
  static constexpr int LD = W + OP::PAD;
  static_assert(NTH % UPR == 0, "whole rows per round");
  Rows rows;
  uint32_t off;  // of round 0
  bool on;       // the thread's columns exist
  u32x4 r[N];
  __device__ __forceinline__ void init(const Rows& t) {
    rows = t;
    on = 16 * (threadIdx.x % UPR) < t.width;
    off = rows.row(threadIdx.x / UPR, OP::C) + 16 * (threadIdx.x % UPR);
  }
  // The next chunk's n rows (rows at or past C, where the threads are more
  // than the units, lie past n).
  __device__ __forceinline__ void load(int n) {
    const rsrc_t b = rows.chunk(n);
    const uint32_t o = off - rows.shift(n, OP::C), step = rows.step(STEP);
#pragma unroll
    for (int u = 0; u < N; ++u) r[u] = __builtin_amdgcn_raw_buffer_load_b128(b, on ? o + u * step : kNone, 0, 0);
    rows.next(OP::C);
  }
  __device__ __forceinline__ void store(typename OP::E* dst) const {
    typename OP::E* p = dst + threadIdx.x / UPR * LD + OP::PER * (threadIdx.x % UPR);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (UNITS % NTH == 0 || u * NTH + static_cast<int>(threadIdx.x) < UNITS)
        *reinterpret_cast<u32x4*>(p + u * STEP * LD) = r[u];
  }
};

constexpr int kW2 = kLinSlice;

// Place of P's element (i, j), j a multiple of 4: rows of C elements without
// gaps, their 16-byte units exchanged by the row's number so that a column of
// units spreads over the LDS banks.
template <typename OP>
__device__ __forceinline__ int p_at(int i, int j) {
  constexpr int U = OP::PER;
  return i * OP::C + ((j / U) ^ (i & (OP::C / U - 1))) * U + j % U;
}

// Decay factors of a chunk's rows.
template <int C>
struct alignas(16) Decay {
  double A[C];             // log2, running
  float fo[C], fz[C];      // 2^A_i, 2^(A_C - A_i)
  float up[C];             // 2^(A_i - A_b), b the first row of i's block of 16
  float down[C];           // 2^(A_b' - A_i), b' the first row of the next block
  float block[C / 16];     // 2^(A_b' - A_b)
  float all;               // 2^A_C
};

// Where a workgroup works.
struct Walk {
  LinChain c;
  int64_t b, bh, seg, row0;  // row0: the segment's first token row
  int64_t t0, len;           // the segment's first token in its sequence, its length
  int h, col0, sl;
  int64_t part0;             // its first partial row
  bool first, last;          // of the sequence's segments, in the chain's direction
};

// What a walk computes.  NS: operands that P and H enter the output's products
// as; EX: the terms e too; WIDE: the output is stored in fp32; ADD: what earlier
// launches left of it, over other value heads, is added.
template <int NS_, bool EX_, bool WIDE_, bool ADD_ = false>
struct Job {
  static constexpr int NS = NS_;
  static constexpr bool EX = EX_, WIDE = WIDE_, ADD = ADD_;
};

template <typename OP, int D1P>
struct Tiles {
  static constexpr int C = OP::C, NI = C / 16, KB = D1P / 32, KS = C / 32, NT = D1P / 16;
  static constexpr int LD1 = D1P + OP::PAD, LDZ = kW2 + OP::PAD;
};

// The rows of an operand of the walk, from the walk's first token on.
template <typename E>
__device__ __forceinline__ Rows walk_rows(const Walk& w, const void* p, int64_t stride, int group, int D, int col,
                                          int width) {
  const int64_t start = w.row0 + (w.c.rev ? w.len - 1 : 0);
  const char* at = static_cast<const char*>(p) +
                   (start * stride + static_cast<int64_t>(w.h / group) * D + col) * static_cast<int64_t>(sizeof(E));
  return Rows{at, static_cast<uint32_t>(stride * sizeof(E)), static_cast<uint32_t>(width * sizeof(E)),
              w.c.rev != 0};
}

// The decays of the walk's chunks, by one wave: lane i reads row i's gate.
struct Gates {
  const float* p;
  int64_t step;
  float g;
  __device__ __forceinline__ void init(const LinChains& a, const Walk& w) {
    const int64_t start = w.row0 + (w.c.rev ? w.len - 1 : 0);
    p = a.g ? a.g + w.h + (a.head_decay ? 0 : start * a.Hv) : nullptr;
    step = a.head_decay ? 0 : w.c.rev ? -a.Hv : a.Hv;
  }
  __device__ __forceinline__ void load(int64_t at, int n) {
    g = p && lane_id() < n ? p[(at + lane_id()) * step] : 0.f;
  }
  // The chunk's factors into d; returns its log2 decay.
  template <int C>
  __device__ __forceinline__ double put(Decay<C>& d, bool rev) const {
    const int lane = lane_id();
    const double g2 = log2_decay(g), inc = prefix64(g2), A = rev ? inc - g2 : inc, all = last_lane(inc);
    const double Ab = row_first(A), next = __shfl(A, ((lane & ~15) + 16) & 63, 64);
    const double An = lane < C - 16 ? next : A;
    if (lane < C) {
      d.A[lane] = A;
      d.fo[lane] = __builtin_amdgcn_exp2f(static_cast<float>(A));
      d.fz[lane] = __builtin_amdgcn_exp2f(static_cast<float>(all - A));
      d.up[lane] = __builtin_amdgcn_exp2f(static_cast<float>(A - Ab));
      const float down = __builtin_amdgcn_exp2f(static_cast<float>(An - A));
      d.down[lane] = down;
      if (lane % 16 == 0) d.block[lane / 16] = down;
    }
    if (lane == 0) d.all = __builtin_amdgcn_exp2f(static_cast<float>(all));
    return all;
  }
};

// Where an output wave stores, 4 columns of a row at a time, and with ADD the
// fp32 rows that it adds.
template <typename J>
struct Out {
  static constexpr uint32_t SIZE = J::WIDE ? 4 : 2;
  Rows o, p;
  __device__ __forceinline__ void init(const LinChains& a, const Walk& w, int w2) {
    const LinChain& c = w.c;
    const bool rev = c.rev != 0;
    const int64_t first = rev ? w.len - 1 : 0, part = w.part0 + first;
    const int heads = a.Hv / c.og, h = w.h / c.og;
    const int64_t row = c.out_partial ? part : w.row0 + first;
    const uint32_t wide = static_cast<uint32_t>(heads) * c.D2;
    o = Rows{static_cast<char*>(c.out) + ((row * heads + h) * c.D2 + w.col0) * SIZE, wide * SIZE, w2 * SIZE, rev};
    if constexpr (J::ADD)
      p = Rows{reinterpret_cast<char*>(c.sum) + ((part * heads + h) * c.D2 + w.col0) * 4, wide * 4,
               static_cast<uint32_t>(w2) * 4, rev};
  }
  // The sum so far at row i, column col (on: inside).
  __device__ __forceinline__ f32x4 before(int n, int C, int i, int col, bool on) const {
    const uint32_t at = p.row(i, C) + col * 4 - p.shift(n, C);
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(p.chunk(n), on ? at : kNone, 0, 0));
  }
  __device__ __forceinline__ void put(int n, int C, int i, int col, bool on, f32x4 v) const {
    const uint32_t at = on ? o.row(i, C) + col * SIZE - o.shift(n, C) : kNone;
    if constexpr (J::WIDE) {
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), o.chunk(n), at, 0, 0);
    } else {
      const bf16x4 q{static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1]), static_cast<__bf16>(v[2]),
                     static_cast<__bf16>(v[3])};
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, q), o.chunk(n), at, 0, 0);
    }
  }
  __device__ __forceinline__ void next(int C) {
    o.next(C);
    if constexpr (J::ADD) p.next(C);
  }
};

// One chunk's update of a state wave's columns: H <- 2^A_C H + Y^T (2^(A_C - A_j) Z).
template <typename OP, int D1P>
__device__ __forceinline__ void update(f32x4 (&H)[D1P / 16], const typename OP::E* Ys, const typename OP::E* Zs,
                                       const Decay<OP::C>& d, int wc) {
  using T = Tiles<OP, D1P>;
  using F = typename OP::F;
  constexpr int NU = OP::FULL, G = T::NT < 8 ? T::NT : 4, STEPS = T::NT / G;
  const int g8 = 8 * (lane_id() >> 4);
  // fragments of Y are read a step ahead of the products that take them, and
  // a step's tiles are independent: the products of one tile wait on each other
  F yt[2][G];
  auto read = [&](int step) {
#pragma unroll
    for (int t = 0; t < G; ++t) {
      const int tile = step % STEPS * G + t;
      yt[step % 2][t] = OP::col(Ys, T::LD1, 32 * (step / STEPS), 32 * (tile / 2) + 4 * (tile % 2), 8);
    }
  };
  read(0);
  F zu[NU];
  const float ft = d.all;
#pragma unroll
  for (int step = 0; step < T::KS * STEPS; ++step) {
    const int ks = step / STEPS, t0 = step % STEPS * G;
    if (step + 1 < T::KS * STEPS) read(step + 1);
    if (t0 == 0) {
      float x[8];
      OP::widen(x, OP::col(Zs, T::LDZ, 32 * ks, wc, 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= d.fz[32 * ks + g8 + i];
      OP::template split<NU>(zu, x);
    }
    if (ks == 0)
#pragma unroll
      for (int t = 0; t < G; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) H[t0 + t][e] *= ft;
#pragma unroll
    for (int s = NU - 1; s >= 0; --s)
#pragma unroll
      for (int t = 0; t < G; ++t) H[t0 + t] = OP::mma(yt[step % 2][t], zu[s], H[t0 + t]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// LDS of a walk: XB buffers of the chunk's rows and HB of H, two of each where
// they fit, so that one chunk's readers do not hold up the next one's writers;
// P and the waves' parts of e where the output waves work by columns.
template <typename OP, int D1P, int NS>
struct Room {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  struct Chunk {
    alignas(16) E X[T::C * T::LD1], Y[T::C * T::LD1], Z[T::C * T::LDZ];
  };
  struct State {
    typename OP::F f[4][T::KB][NS][64];  // [16 columns][32 rows][operand][lane]
  };
  static constexpr bool COLS = NS > 2;
  struct Rest {
    Decay<T::C> d[COLS ? 1 : 2];
    alignas(16) E P[COLS ? NS * T::C * T::C : 8];
    float e[COLS ? 4 : 1][T::C];
  };
  static constexpr size_t kMax = 160 * 1024 - sizeof(Rest);
  static constexpr int XB = 2 * sizeof(Chunk) + sizeof(State) <= kMax ? 2 : 1;
  static constexpr int HB = XB == 2 && 2 * sizeof(Chunk) + 2 * sizeof(State) <= kMax && !COLS ? 2 : 1;
  struct Buffers : Rest {
    Chunk x[XB];
    State h[HB];
  };
};

// H for the output waves, as NS operands.
template <typename OP, int D1P, int NS, typename S>
__device__ __forceinline__ void hand_over(const f32x4 (&H)[D1P / 16], S& s, int cg) {
#pragma unroll
  for (int kb = 0; kb < D1P / 32; ++kb) {
    const f32x4 h0 = H[2 * kb], h1 = H[2 * kb + 1];
    const float x[8] = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
    typename OP::F f[NS];
    OP::template split<NS>(f, x);
#pragma unroll
    for (int k = 0; k < NS; ++k) s.f[cg][kb][k][lane_id()] = f[k];
  }
}

// The rows of a walk's chunks on their way through registers to LDS (by all
// eight waves), and the gates (by one).
template <typename OP, int D1P, typename R>
struct Feed {
  using E = typename OP::E;
  static constexpr int C = OP::C;
  Stage<OP, D1P, 512> x, y;
  Stage<OP, kW2, 512> z;
  Gates g;
  int64_t len;
  bool mine, rev;
  __device__ __forceinline__ void init(const LinChains& a, const Walk& w, int wave) {
    const LinChain& c = w.c;
    x.init(walk_rows<E>(w, c.x, c.xr, c.xg, c.D1, 0, c.D1));
    y.init(walk_rows<E>(w, c.y, c.yr, c.yg, c.D1, 0, c.D1));
    z.init(walk_rows<E>(w, c.z, c.zr, c.zg, c.D2, w.col0, min(c.D2 - w.col0, kW2)));
    g.init(a, w);
    len = w.len, rev = c.rev;
    mine = wave == (R::COLS ? 7 : 1);  // by rows, 16 .. 31 are little work
  }
  __device__ __forceinline__ int rows(int64_t at) const {
    return static_cast<int>(min(len - at, static_cast<int64_t>(C)));
  }
  // Loads the chunk at `at`, if there is one.
  __device__ __forceinline__ void fetch(int64_t at) {
    if (at >= len) return;
    const int n = rows(at);
    x.load(n);
    y.load(n);
    z.load(n);
  }
  __device__ __forceinline__ void put(typename R::Chunk& to) const {
    x.store(to.X);
    y.store(to.Y);
    z.store(to.Z);
  }
  // The decays of the chunk whose gates are loaded, and loads the next one's.
  __device__ __forceinline__ void decays(Decay<C>& d, int64_t next) {
    if (!mine) return;
    g.put(d, rev);
    if (next < len) g.load(next, rows(next));
  }
};

// What a walk does around each chunk's work.  With two buffers of both kinds a
// chunk takes one barrier: its readers work while the next chunk's rows are
// written (loaded a chunk before) and the state waves hand the next H over.
// With one buffer of H the state waves hand it over between two barriers,
// behind its last reader; with one buffer of the rows these are loaded as the
// chunk's work starts and written between the barriers too.
template <typename OP, int D1P, typename R>
__device__ __forceinline__ void walk_start(Feed<OP, D1P, R>& f, typename R::Buffers& s) {
  f.fetch(0);
  if (f.mine) f.g.load(0, f.rows(0));
  f.decays(s.d[0], OP::C);
  f.put(s.x[0]);
  if constexpr (R::XB == 2) f.fetch(OP::C);
}
template <typename OP, int D1P, typename R>
__device__ __forceinline__ void chunk_start(Feed<OP, D1P, R>& f, typename R::Buffers& s, int64_t at, int b) {
  if (at + OP::C >= f.len) return;
  if constexpr (R::XB == 2) {
    f.put(s.x[b ^ 1]);
    f.fetch(at + 2 * OP::C);
  } else {
    f.fetch(at + OP::C);
  }
  if constexpr (!R::COLS) f.decays(s.d[b ^ 1], at + 2 * OP::C);
}
template <typename OP, int D1P, typename R>
__device__ __forceinline__ void chunk_end(Feed<OP, D1P, R>& f, typename R::Buffers& s, int64_t at) {
  if (at + OP::C >= f.len) return;
  if constexpr (R::XB == 1) f.put(s.x[0]);
  if constexpr (R::COLS) f.decays(s.d[0], at + 2 * OP::C);
}

// The state waves' part of a walk.
template <typename OP, int D1P, typename R, int NS>
__device__ __forceinline__ void carry_state(f32x4 (&H)[D1P / 16], Feed<OP, D1P, R>& f, typename R::Buffers& s, int cg) {
  constexpr int C = OP::C;
  hand_over<OP, D1P, NS>(H, s.h[0], cg);
  __syncthreads();
  int b = 0;
  for (int64_t at = 0; at < f.len; at += C, b ^= 1) {
    chunk_start(f, s, at, b);
    const auto& x = s.x[R::XB == 2 ? b : 0];
    update<OP, D1P>(H, x.Y, x.Z, s.d[R::COLS ? 0 : b], 16 * cg);
    if constexpr (R::HB == 1) __syncthreads();
    chunk_end(f, s, at);
    if (at + C < f.len) hand_over<OP, D1P, NS>(H, s.h[R::HB == 2 ? b ^ 1 : 0], cg);
    __syncthreads();
  }
}

// The output waves' part, a wave forming 16 rows of a chunk: X H and P of its
// rows, and P Z from registers, without a barrier between.
template <typename OP, int D1P, typename R, typename J>
__device__ __forceinline__ void out_by_rows(const LinChains& a, const Walk& w, Feed<OP, D1P, R>& f,
                                            typename R::Buffers& s, int wave) {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  using F = typename OP::F;
  constexpr int C = T::C, NI = T::NI, KB = T::KB, KS = T::KS, NS = J::NS;
  constexpr bool EX = J::EX;
  constexpr uint32_t ES = sizeof(E);
  const LinChain& c = w.c;
  const int lane = lane_id(), m = lane & 15, g4 = 4 * (lane >> 4), w2 = min(c.D2 - w.col0, kW2);
  const bool rev = c.rev;
  // The wave's 16 rows of a chunk and its NI tiles of 16 columns.
  const int ib = wave % NI, ct0 = wave / NI * NI, i = 16 * ib + m;
  Out<J> out;
  out.init(a, w, w2);
  Rows re{};
  uint32_t oe = 0;
  if constexpr (EX) {
    re = walk_rows<E>(w, c.ex, c.er, c.eg, c.D2, w.col0, w2);
    oe = re.row(i, C) + g4 * ES;
  }
  // e in parts: a wave sums its NI tiles of columns
  float* const ep =
      EX ? c.e + (static_cast<int64_t>(w.sl * (4 / NI) + wave / NI) * a.Hv + w.h) * a.rows + w.part0 : nullptr;
  __syncthreads();

  int b = 0;
  for (int64_t at = 0; at < w.len; at += C, b ^= 1) {
    const int n = f.rows(at);
    chunk_start(f, s, at, b);
    const auto& x = s.x[R::XB == 2 ? b : 0];
    const auto& h = s.h[R::HB == 2 ? b : 0];
    const auto& d = s.d[R::COLS ? 0 : b];
    float ex[NI][4];
    if constexpr (EX) {
      const rsrc_t be = re.chunk(n);
      const uint32_t at0 = oe - re.shift(n, C);
      re.next(C);
#pragma unroll
      for (int t = 0; t < NI; ++t) {
        const int col = 16 * (ct0 + t);
        const uint32_t o = col < w2 ? at0 + col * ES : kNone;
        if constexpr (ES == 2) {
          const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(be, o, 0, 0);
          ex[t][0] = __uint_as_float(u[0] << 16), ex[t][1] = __uint_as_float(u[0] & 0xffff0000u);
          ex[t][2] = __uint_as_float(u[1] << 16), ex[t][3] = __uint_as_float(u[1] & 0xffff0000u);
        } else {
          const u32x4 u = __builtin_amdgcn_raw_buffer_load_b128(be, o, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) ex[t][e] = __uint_as_float(static_cast<unsigned>(u[e]));
        }
      }
    }

    f32x4 pv[NI];
    if constexpr (J::ADD)
#pragma unroll
      for (int t = 0; t < NI; ++t) pv[t] = out.before(n, C, i, 16 * (ct0 + t) + g4, 16 * (ct0 + t) < w2);

    // X H of the wave's rows, transposed; fragments are read a step ahead of
    // the products that take them
    f32x4 O[NI];
#pragma unroll
    for (int t = 0; t < NI; ++t) O[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    F xf[KB], hf[2][NI][NS];
    auto read = [&](int kb) {
      xf[kb] = OP::run(x.X + i * T::LD1 + 32 * kb + 2 * g4);
#pragma unroll
      for (int t = 0; t < NI; ++t)
#pragma unroll
        for (int q = 0; q < NS; ++q) hf[kb % 2][t][q] = h.f[ct0 + t][kb][q][lane];
    };
    read(0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 1 < KB) read(kb + 1);
#pragma unroll
      for (int q = NS - 1; q >= 0; --q)
#pragma unroll
        for (int t = 0; t < NI; ++t) O[t] = OP::mma(hf[kb % 2][t][q], xf[kb], O[t]);
      __builtin_amdgcn_sched_barrier(0);
    }
    const float fo = d.fo[i], up = d.up[i];
    const double Ai = d.A[i];
#pragma unroll
    for (int t = 0; t < NI; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) O[t][e] *= fo;

    // 32 columns of P at a time, transposed (the lane holds columns j .. j + 3
    // of row i in each of two tiles), and O += P Z from them.  On the diagonal
    // tile each factor 2^(A_i - A_j) is formed from its difference; below, it
    // is 2^(A_i - A_b) 2^(A_b - A_b') 2^(A_b' - A_j), b the wave's first row and
    // b' that of the block after j's.
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      if (2 * ks <= ib) {
        f32x4 S2[2] = {f32x4{0.f, 0.f, 0.f, 0.f}, f32x4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            S2[t] = OP::mma(OP::run(x.Y + (32 * ks + 16 * t + m) * T::LD1 + 32 * kb + 2 * g4), xf[kb], S2[t]);
        F zf[NI];
#pragma unroll
        for (int t = 0; t < NI; ++t) zf[t] = OP::pair(x.Z, T::LDZ, 32 * ks, 16 * (ct0 + t));
        float p[8];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int jb = 2 * ks + t, j = 16 * jb + g4;
          if (jb < ib) {
            const f32x4 df = *reinterpret_cast<const f32x4*>(&d.down[j]);
            float u = up;
            for (int k = jb + 1; k < ib; ++k) u *= d.block[k];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[4 * t + e] = S2[t][e] * (u * df[e]);
          } else if (jb == ib) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[4 * t + e] =
                  j + e <= i ? S2[t][e] * __builtin_amdgcn_exp2f(static_cast<float>(Ai - d.A[j + e])) : 0.f;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) p[4 * t + e] = 0.f;
          }
        }
        F pf[NS];
        OP::template split<NS>(pf, p);
#pragma unroll
        for (int q = NS - 1; q >= 0; --q)
#pragma unroll
          for (int t = 0; t < NI; ++t) O[t] = OP::mma(zf[t], pf[q], O[t]);
      }

    float e = 0.f;
#pragma unroll
    for (int t = 0; t < NI; ++t) {
      const f32x4 v = O[t];
      const int col = 16 * (ct0 + t);
      if constexpr (EX) e += (ex[t][0] * v[0] + ex[t][1] * v[1]) + (ex[t][2] * v[2] + ex[t][3] * v[3]);
      if constexpr (J::ADD) out.put(n, C, i, col + g4, col < w2, v + pv[t]);
      else out.put(n, C, i, col + g4, col < w2, v);
    }
    out.next(C);
    if constexpr (EX) {
      e = rows4_sum(e);
      const int64_t row = rev ? w.len - 1 - at - i : at + i;
      if (lane < 16 && i < n) ep[row] = e;
    }
    if constexpr (R::HB == 1) __syncthreads();
    chunk_end(f, s, at);
    __syncthreads();
  }
}

// The output waves' part, a wave forming 16 columns: it reads the operands of
// its columns of H alone, which matters where H is three operands; the waves'
// column blocks of P pass through LDS.
template <typename OP, int D1P, typename R, typename J>
__device__ __forceinline__ void out_by_columns(const LinChains& a, const Walk& w, Feed<OP, D1P, R>& f,
                                               typename R::Buffers& s, int wave) {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  using F = typename OP::F;
  constexpr int C = T::C, NI = T::NI, KB = T::KB, KS = T::KS, NS = J::NS;
  constexpr bool EX = J::EX;
  constexpr uint32_t ES = sizeof(E);
  const LinChain& c = w.c;
  const int tid = threadIdx.x, lane = lane_id(), m = lane & 15, g4 = 4 * (lane >> 4), w2 = min(c.D2 - w.col0, kW2);
  const bool rev = c.rev;
  const int wc = 16 * wave;  // the wave's first column in the slice
  Out<J> out;
  out.init(a, w, w2);
  Rows re{};
  uint32_t oe = 0;
  if constexpr (EX) {
    re = walk_rows<E>(w, c.ex, c.er, c.eg, c.D2, w.col0, w2);
    oe = re.row(m, C) + (wc + g4) * ES;
  }
  const bool has = wc < w2;
  // the wave's column block of P, and the row blocks in the order it takes them
  const int jb = wave % NI;
  int blk[NI];
#pragma unroll
  for (int k = 0; k < NI; ++k) blk[k] = (jb + k) % NI;
  __syncthreads();

  int b = 0;
  for (int64_t at = 0; at < w.len; at += C, b ^= 1) {
    const int n = f.rows(at);
    chunk_start(f, s, at, b);
    const auto& x = s.x[R::XB == 2 ? b : 0];
    const auto& h = s.h[0];
    const auto& d = s.d[R::COLS ? 0 : b];
    // X H, and the wave's block of P; both transposed.  Fragments are read a
    // step ahead of the products that take them.
    f32x4 O[NI], S4[NI];
#pragma unroll
    for (int k = 0; k < NI; ++k) O[k] = S4[k] = f32x4{0.f, 0.f, 0.f, 0.f};
    F xf[2][NI], yf[2], hf[2][NS];
    auto read = [&](int kb) {
      yf[kb % 2] = OP::run(x.Y + (16 * jb + m) * T::LD1 + 32 * kb + 2 * g4);
#pragma unroll
      for (int k = 0; k < NS; ++k) hf[kb % 2][k] = h.f[wave][kb][k][lane];
#pragma unroll
      for (int k = 0; k < NI; ++k) xf[kb % 2][k] = OP::run(x.X + (16 * blk[k] + m) * T::LD1 + 32 * kb + 2 * g4);
    };
    read(0);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      if (kb + 1 < KB) read(kb + 1);
#pragma unroll
      for (int k = 0; k < NI; ++k) S4[k] = OP::mma(yf[kb % 2], xf[kb % 2][k], S4[k]);
#pragma unroll
      for (int q = NS - 1; q >= 0; --q)
#pragma unroll
        for (int k = 0; k < NI; ++k) O[k] = OP::mma(hf[kb % 2][q], xf[kb % 2][k], O[k]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // P = S o 2^(A_i - A_j): the lane holds rows j .. j + 3 of column i; the
    // factors as in out_by_rows
    if (NI == 4 || wave < NI) {
      const int j = 16 * jb + g4;
      f32x4 df = *reinterpret_cast<const f32x4*>(&d.down[j]);
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const int i = 16 * blk[k] + m;
        f32x4 p;
        if (k == 0) {
          const double Ai = d.A[i];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[e] = j + e <= i ? S4[k][e] * __builtin_amdgcn_exp2f(static_cast<float>(Ai - d.A[j + e])) : 0.f;
        } else {
          const bool below = jb + k < NI;
          const float u = d.up[i], bl = d.block[blk[k]];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = below ? S4[k][e] * (u * df[e]) : 0.f;
            df[e] *= bl;
          }
        }
        OP::template put4<NS>(s.P + p_at<OP>(i, j), C * C, p);
      }
    }
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const float fo = d.fo[16 * blk[k] + m];
#pragma unroll
      for (int e = 0; e < 4; ++e) O[k][e] *= fo;
    }
    F zf[KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) zf[ks] = OP::col(x.Z, T::LDZ, 32 * ks, wc, 4);
    f32x4 pv[NI];
    if constexpr (J::ADD)
#pragma unroll
      for (int k = 0; k < NI; ++k) pv[k] = out.before(n, C, 16 * blk[k] + m, wc + g4, has);
    float ex[NI][4];
    if constexpr (EX) {
      const rsrc_t be = re.chunk(n);
      const uint32_t step = re.step(16), at0 = oe - re.shift(n, C);
      re.next(C);
#pragma unroll
      for (int k = 0; k < NI; ++k) {
        const uint32_t o = has ? at0 + blk[k] * step : kNone;
        if constexpr (ES == 2) {
          const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(be, o, 0, 0);
          ex[k][0] = __uint_as_float(u[0] << 16), ex[k][1] = __uint_as_float(u[0] & 0xffff0000u);
          ex[k][2] = __uint_as_float(u[1] << 16), ex[k][3] = __uint_as_float(u[1] & 0xffff0000u);
        } else {
          const u32x4 u = __builtin_amdgcn_raw_buffer_load_b128(be, o, 0, 0);
#pragma unroll
          for (int e = 0; e < 4; ++e) ex[k][e] = __uint_as_float(static_cast<unsigned>(u[e]));
        }
      }
    }
    __syncthreads();

    // O += P Z; the blocks of P above the diagonal are zeros
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int q = NS - 1; q >= 0; --q) {
        F pf[NI];
#pragma unroll
        for (int k = 0; k < NI; ++k) pf[k] = OP::prun(s.P + q * C * C, 16 * blk[k] + m, 32 * ks + 2 * g4);
#pragma unroll
        for (int k = 0; k < NI; ++k) O[k] = OP::mma(zf[ks], pf[k], O[k]);
      }
    chunk_end(f, s, at);
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      const f32x4 v = O[k];
      if constexpr (J::ADD) out.put(n, C, 16 * blk[k] + m, wc + g4, has, v + pv[k]);
      else out.put(n, C, 16 * blk[k] + m, wc + g4, has, v);
      if constexpr (EX) {
        const float e = rows4_sum((ex[k][0] * v[0] + ex[k][1] * v[1]) + (ex[k][2] * v[2] + ex[k][3] * v[3]));
        if (lane < 16) s.e[wave][16 * blk[k] + m] = e;
      }
    }
    out.next(C);
    __syncthreads();
    if constexpr (EX) {
      if (tid < n) {
        const int64_t row = w.part0 + (rev ? w.len - 1 - at - tid : at + tid);
        c.e[(static_cast<int64_t>(w.sl) * a.Hv + w.h) * a.rows + row] = (s.e[0][tid] + s.e[1][tid]) + (s.e[2][tid] + s.e[3][tid]);
      }
    }
  }
}

// One walk over a segment of at least one token; H: the state waves' columns.
template <typename OP, int D1P, typename R, typename J>
__device__ __forceinline__ void walk(const LinChains& a, const Walk& w, f32x4 (&H)[D1P / 16], typename R::Buffers& s) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Feed<OP, D1P, R> f;
  f.init(a, w, wave);
  walk_start(f, s);
  if (wave >= 4) carry_state<OP, D1P, R, J::NS>(H, f, s, wave & 3);
  else if constexpr (R::COLS) out_by_columns<OP, D1P, R, J>(a, w, f, s, wave);
  else out_by_rows<OP, D1P, R, J>(a, w, f, s, wave);
}

// The launch's units of work: one chain, slice, segment, sequence and value
// head each, or, in a sum over heads, key head (and the launch's value head of
// it).  Those of the dq and dk chains come first: they take longest.  Within either kind slices are fastest, then
// the value heads that share a key head, then sequences, then segments, then
// key heads; and each of the 8 XCDs takes a contiguous range, so that units
// that read the same rows share an L2, and as much of it as the others,
// whatever the sequences' lengths.
struct Units {
  int64_t early, late;  // per XCD
};
__host__ __device__ inline Units units(const LinChains& a) {
  int n = 0, keys = 0;
  for (int i = 0; i < a.n; ++i) (a.c[i].key ? keys : n) += lin_slices(a.c[i].D2);
  const int64_t heads = a.B * a.Hv * a.segments;
  const int64_t early = keys * (a.sum ? heads / a.group : heads), late = n * heads;
  return Units{(early + 7) / 8, (late + 7) / 8};
}

// Finds the workgroup's unit; false: nothing to do.
__device__ __forceinline__ bool find(const LinChains& a, const Units& u, int64_t block, Walk& w) {
  const int64_t xcd = block % 8, k = block / 8;
  const bool early = k < u.early;
  const int64_t index = early ? xcd * u.early + k : xcd * u.late + k - u.early;
  const int first = early || a.n < 3 ? 0 : 2, end = early ? 2 : a.n;
  const int n0 = lin_slices(a.c[first == 2 ? 2 : 0].D2), all = n0 + (end - first > 1 ? lin_slices(a.c[1].D2) : 0);
  int s = static_cast<int>(index % all);
  int64_t r = index / all;
  const int group = early && a.sum ? 1 : a.group, heads = early && a.sum ? a.Hv / a.group : a.Hv;
  if (r >= a.B * heads * a.segments) return false;
  const int ci = s < n0 ? first : first + 1;
  s -= ci == first ? 0 : n0;
  w.c = lin_chain(ci);
  w.sl = s;
  w.col0 = s * kW2;
  const int64_t per = group * a.B;
  w.b = r % per / group;
  w.seg = r / per % a.segments;
  w.h = static_cast<int>(r / (per * a.segments)) * group + static_cast<int>(r % group);
  if (early && a.sum) w.h = w.h * a.group + a.head;
  w.bh = w.b * a.Hv + w.h;
  const LinSpan sp = lin_span(a.cu, w.b, a.T);
  w.t0 = w.seg * a.seg;
  if (w.t0 >= sp.len && w.seg > 0) return false;
  w.len = min(a.seg, sp.len - w.t0);
  w.row0 = sp.t0 + w.t0;
  w.part0 = lin_part_row(a, w.b, sp, w.t0);
  const bool begin = w.seg == 0, last = w.t0 + w.len >= sp.len;
  w.first = w.c.rev ? last : begin;
  w.last = w.c.rev ? begin : last;
  return true;
}

// The state's elements that a state wave's lane holds: tile t's are rows d1 ..
// d1 + 3 of one column.
template <int D1P, typename F>
__device__ __forceinline__ void each_state(const LinChain& c, int col0, F&& f) {
  const int lane = lane_id(), d2 = col0 + 16 * static_cast<int>(threadIdx.x >> 6 & 3) + (lane & 15);
#pragma unroll
  for (int t = 0; t < D1P / 16; ++t) {
    const int d1 = 32 * (t / 2) + 8 * (lane >> 4) + 4 * (t % 2);
    if (d2 < c.D2 && d1 < c.D1) f(t, static_cast<int64_t>(d1) * c.s1 + static_cast<int64_t>(d2) * c.s2);
  }
}

// A unit's state waves load the state it starts from.
template <int D1P>
__device__ __forceinline__ void load_state(const LinChains& a, const Walk& w, f32x4 (&H)[D1P / 16]) {
  const LinChain& c = w.c;
  const int64_t one = static_cast<int64_t>(c.D1) * c.D2;
#pragma unroll
  for (int t = 0; t < D1P / 16; ++t) H[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* in = c.seg_in ? c.seg_in + (w.bh * a.segments + w.seg) * one : c.s_in ? c.s_in + w.bh * one : nullptr;
  if (in)
    each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
      for (int e = 0; e < 4; ++e) H[t][e] = in[at + static_cast<int64_t>(e) * c.s1];
    });
}

// What they leave at its end: <state, dot> and the state.
template <int D1P>
__device__ __forceinline__ void leave_state(const LinChains& a, const Walk& w, const f32x4 (&H)[D1P / 16]) {
  const LinChain& c = w.c;
  const int64_t one = static_cast<int64_t>(c.D1) * c.D2;
  if (c.xdot) {
    const float* dot = c.seg_dot ? c.seg_dot + (w.bh * a.segments + w.seg) * one : c.dot ? c.dot + w.bh * one : nullptr;
    float x = 0.f;
    if (dot)
      each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x += H[t][e] * dot[at + static_cast<int64_t>(e) * c.s1];
      });
    x = rows4_sum(row16_sum(x));
    if (lane_id() == 0)
      c.xdot[((w.seg * a.B * a.Hv + w.bh) * lin_slices(c.D2) + w.sl) * 4 + (threadIdx.x >> 6 & 3)] = x;
  }
  if (c.s_out && w.last) {
    float* out = c.s_out + w.bh * one;
    each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[at + static_cast<int64_t>(e) * c.s1] = H[t][e];
    });
  }
}

// JA: the job of the dq and dk chains, JB: that of the others.
template <typename OP, int D1P, typename JA, typename JB>
__global__ __launch_bounds__(512) void lin_chunk_kernel(LinChains a, Units u) {
  constexpr int NS = JA::NS > JB::NS ? JA::NS : JB::NS;
  using R = Room<OP, D1P, NS>;
  __shared__ typename R::Buffers s;
  const bool state = threadIdx.x >= 256;
  f32x4 H[D1P / 16];
  int64_t block = blockIdx.x;
  {
    Walk w;
    if (!find(a, u, block, w)) return;
    if (state) load_state<D1P>(a, w, H);
    if (w.len > 0) {
      if (!std::is_same_v<JA, JB> && w.c.key) walk<OP, D1P, R, JA>(a, w, H, s);
      else walk<OP, D1P, R, JB>(a, w, H, s);
    }
  }
  if (!state) return;
  // the unit is found again: kept over the walk, it would crowd the walk's
  // own scalars out of their registers
  asm volatile("" : "+s"(block));
  Walk w;
  find(a, u, block, w);
  leave_state<D1P>(a, w, H);
}

// Every segment's own contribution to the state at its end (in the chain's
// direction), from zero, by four state waves.  The last segment's is not
// needed.  The chain forward in time leaves the segments' factors, but the
// last one's, which only the chain backward in time needs and leaves.  Measured
// at 32768 tokens of 8 heads in 32 segments: 45 us, the scan 17, the walks 90.
template <typename OP, int D1P>
__global__ __launch_bounds__(256) void lin_segment_kernel(LinChains a, Units u, float* factor) {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  constexpr int C = T::C;
  __shared__ __align__(16) E Ys[C * T::LD1], Zs[C * T::LDZ];
  __shared__ __align__(16) Decay<C> d;
  Walk w;
  if (!find(a, u, blockIdx.x, w) || w.last) return;
  const LinChain& c = w.c;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w2 = min(c.D2 - w.col0, kW2);
  f32x4 H[D1P / 16];
#pragma unroll
  for (int t = 0; t < D1P / 16; ++t) H[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  Stage<OP, D1P, 256> sy;
  Stage<OP, kW2, 256> sz;
  sy.init(walk_rows<E>(w, c.y, c.yr, c.yg, c.D1, 0, c.D1));
  sz.init(walk_rows<E>(w, c.z, c.zr, c.zg, c.D2, w.col0, w2));
  Gates gates;
  gates.init(a, w);
  double total = 0.0;
  auto fetch = [&](int64_t at) {
    const int n = static_cast<int>(min(w.len - at, static_cast<int64_t>(C)));
    sy.load(n);
    sz.load(n);
    if (wave == 3) gates.load(at, n);
  };
  fetch(0);
  for (int64_t at = 0; at < w.len; at += C) {
    sy.store(Ys);
    sz.store(Zs);
    if (wave == 3) total += gates.put(d, c.rev);
    __syncthreads();
    if (at + C < w.len) fetch(at + C);
    update<OP, D1P>(H, Ys, Zs, d, 16 * wave);
    __syncthreads();
  }
  const int64_t at0 = w.bh * a.segments + w.seg, one = static_cast<int64_t>(c.D1) * c.D2;
  if ((!c.rev || w.first) && w.sl == 0 && threadIdx.x == 192)
    factor[at0] = __builtin_amdgcn_exp2f(static_cast<float>(total));
  float* out = c.s_out + at0 * one;
  each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[at + static_cast<int64_t>(e) * c.s1] = H[t][e];
  });
}

// Segment states in place: what each segment starts from.  blockIdx.y:
// forward in time from h0, backward from dht.  A thread takes 4 elements of
// one (b, v-head) through all its segments.
__global__ __launch_bounds__(256) void lin_scan_kernel(float* fwd, float* rev, const float* factor, const float* h0,
                                                       const float* dht, int one, int64_t BH, int Hv, int64_t T,
                                                       int64_t segments, int64_t seg, const int64_t* cu) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t bh = i / (one / 4);
  if (bh >= BH) return;
  const int64_t at = i % (one / 4) * 4;
  const bool back = blockIdx.y;
  float* S = (back ? rev : fwd) + bh * segments * one + at;
  const float* init = back ? dht : h0;
  const int64_t len = lin_span(cu, bh / Hv, T).len, n = len > 0 ? (len + seg - 1) / seg : 1;
  f32x4 cur{0.f, 0.f, 0.f, 0.f};
  if (init) cur = *reinterpret_cast<const f32x4*>(init + bh * one + at);
  for (int64_t k = 0; k < n; ++k) {
    const int64_t s = back ? n - 1 - k : k;
    const f32x4 own = *reinterpret_cast<const f32x4*>(S + s * one);
    *reinterpret_cast<f32x4*>(S + s * one) = cur;
    const float f = factor[bh * segments + s];
#pragma unroll
    for (int e = 0; e < 4; ++e) cur[e] = f * cur[e] + own[e];
  }
}

int max_d1(const LinChains& a) {
  int d = 0;
  for (int i = 0; i < a.n; ++i) d = std::max(d, a.c[i].D1);
  return d;
}

template <typename OP, int D1P, typename JA, typename JB = JA>
hipError_t run_chunks(const LinChains& a, hipStream_t st) {
  const Units u = units(a);
  lin_chunk_kernel<OP, D1P, JA, JB><<<static_cast<unsigned>(8 * (u.early + u.late)), 512, 0, st>>>(a, u);
  return hipGetLastError();
}

template <typename OP, int D1P>
hipError_t run_segments(const LinChains& a, float* factor, hipStream_t st) {
  const Units u = units(a);
  lin_segment_kernel<OP, D1P><<<static_cast<unsigned>(8 * (u.early + u.late)), 256, 0, st>>>(a, u, factor);
  return hipGetLastError();
}

// The kernel of a VJP: whether e is wanted, dv is returned in fp32, dq and dk
// are stored in fp32 in any case (`part`), and added to what is there (`add`).
template <typename OP, int D1P, bool WIDE>
hipError_t run_vjp(const LinChains& a, bool ex, bool add, bool part, hipStream_t st) {
  constexpr int N = OP::FULL, M = WIDE ? N : OP::NARROW;  // operands with e, without
  using JB = Job<M, false, WIDE>;
  if (add && (part || WIDE)) return ex ? run_chunks<OP, D1P, Job<N, true, true, true>, JB>(a, st)
                                       : run_chunks<OP, D1P, Job<M, false, true, true>, JB>(a, st);
  if (add) return ex ? run_chunks<OP, D1P, Job<N, true, WIDE, true>, JB>(a, st)
                     : run_chunks<OP, D1P, Job<M, false, WIDE, true>, JB>(a, st);
  if (part || WIDE) return ex ? run_chunks<OP, D1P, Job<N, true, true>, JB>(a, st)
                              : run_chunks<OP, D1P, Job<M, false, true>, JB>(a, st);
  return ex ? run_chunks<OP, D1P, Job<N, true, WIDE>, JB>(a, st) : run_chunks<OP, D1P, Job<M, false, WIDE>, JB>(a, st);
}

// Calls f with the operand type and the padded width (an integral constant).
// 256 rows of state leave LDS for chunks of 32 rows only.
template <typename F>
hipError_t by_type(bool io_bf16, int d1, F&& f) {
  constexpr std::integral_constant<int, 64> w64{};
  constexpr std::integral_constant<int, 128> w128{};
  constexpr std::integral_constant<int, 256> w256{};
  if (!io_bf16) return d1 <= 64 ? f(OpF{}, w64) : d1 <= 128 ? f(OpF{}, w128) : f(OpF{}, w256);
  return d1 <= 64 ? f(OpB<64>{}, w64) : d1 <= 128 ? f(OpB<64>{}, w128) : f(OpB<32>{}, w256);
}

}  // namespace

// Cutting sequences.  A workgroup walks a segment's tokens one chunk after
// another and a compute unit holds one workgroup, so a launch takes rounds of
// 256 of them.  More segments fill the last round, or the only one, but cost a
// pass that forms their states; a launch for each value head of a key head saves
// the sum over them, but has fewer workgroups.  The plan with the
// least estimated time is taken, from what was measured on MI355X in bf16 at D =
// 128 (ns a token of a walk), for all types and widths:
//   a walk 45 (forward), 54 (VJP: 768 workgroups of 4096 tokens 654-664 us), and
//   4 us to begin and end;
//   the segment pass 29 with one workgroup on a compute unit, 15 more for each
//   further one (16 segments of 2048 tokens 59 us, 32 of 1024 45 us);
//   the scan 4 us, 0.3 us a segment and its states both ways at 4 TB/s;
//   the sum over heads 5 us and 5.5 TB/s, a further launch 3 us.
// What the rule chose, against the other side: VJP of 4 x 4096 tokens, 16 key
// and 32 value heads, summed by launches 675-690 us, with the sum's pass 752-756;
// of 1 x 4096 tokens, summed and in 4 segments 237-241, whole with the pass
// 262-264; of 16384 tokens of 8 heads 235-238 in 16 segments, 274-276 in 11, 903
// whole; forward of 333 tokens, fp32, 22 in segments of 64, 35 of 192; of 4 x 4096
// tokens 172-176 whole, 250 cut.  Over every cut of 777 .. 16384 tokens of 4 and 8
// heads, forward and VJP, with and without shared key heads: the one chosen takes
// at most 1.12 times the best one's time in bf16 (D = 32, 64, 128, 256) and 1.10
// in fp32 (64, 128).
LinPlan lin_plan(const LinShape& s, bool backward) {
  LinPlan best{};
  double least = 0.0;
  const double bh = static_cast<double>(std::max<int64_t>(1, s.B * s.Hv)), bk = bh * s.Hk / s.Hv, group = s.Hv / s.Hk;
  const double keys = backward ? 2.0 * lin_slices(s.Dk) : 0.0, rest = lin_slices(s.Dv);
  const double token = backward ? 54e-3 : 45e-3;  // us
  auto rounds = [](double n) { return std::ceil(n / 256.0); };
  int64_t seg_before = 0;
  for (int64_t n = 1; n <= 256; n += (n + 7) / 8) {
    const int64_t seg = std::max<int64_t>(64, ((s.T + n - 1) / n + 63) / 64 * 64);
    if (seg == seg_before) continue;
    seg_before = seg;
    const int64_t segments = std::max<int64_t>(1, (s.T + seg - 1) / seg);
    const double m = static_cast<double>(segments), walk = 4.0 + seg * token, ways = backward ? 2.0 : 1.0;
    double pre = 0.0;
    if (segments > 1)
      pre = seg * (29e-3 + 15e-3 * (rounds(ways * bh * rest * m) - 1)) + 4.0 + 0.3 * m +
            2e-6 * ways * bh * m * s.Dk * s.Dv * sizeof(float) / 4.0;
    for (int sum = 0; sum <= (backward && group > 1 ? 1 : 0); ++sum) {
      double us = pre;
      if (sum) us += (walk * rounds(bk * keys * m) + 3.0) * (group - 1) + walk * rounds((bk * keys + bh * rest) * m);
      else us += walk * rounds(bh * (keys + rest) * m);
      if (backward && group > 1 && !sum) us += 5.0 + 1e-6 * bh * s.T * s.Dk * 16.0 / 5.5;
      if (best.segments == 0 || us < least) {
        least = us;
        best.segments = segments, best.seg = seg, best.sum = sum != 0;
      }
    }
    if (seg == 64) break;
  }
  if (best.segments > 1) {
    const size_t n = static_cast<size_t>(s.B) * s.Hv * best.segments;
    best.states = n * s.Dk * s.Dv * sizeof(float);
    best.bytes = (backward ? 2 : 1) * best.states + (n * sizeof(float) + 255) / 256 * 256;
  }
  return best;
}

// One direction's segment states, then their factors.
LinSegs lin_segs(const LinPlan& p, bool backward, char* base) {
  LinSegs g{};
  if (p.segments == 1) return g;
  g.fwd = reinterpret_cast<float*>(base);
  g.rev = backward ? reinterpret_cast<float*>(base + p.states) : nullptr;
  g.factor = reinterpret_cast<float*>(base + (backward ? 2 : 1) * p.states);
  return g;
}

namespace {

// What each segment starts from: the segments' own states, then the scan.
hipError_t segment_states(const LinShape& s, const LinPlan& p, const LinSegs& g, LinChains a, const float* h0,
                          const float* dht, hipStream_t st) {
  a.segments = p.segments, a.seg = p.seg;
  {
    ProfScope prof("linear_segments", st);
    hipError_t e = by_type(s.io_bf16, max_d1(a), [&](auto op, auto d1) {
      return run_segments<decltype(op), decltype(d1)::value>(a, g.factor, st);
    });
    if (e != hipSuccess) return e;
  }
  ProfScope prof("linear_scan", st);
  const int one = s.Dk * s.Dv;
  const int64_t n = s.B * s.Hv * (one / 4);
  lin_scan_kernel<<<dim3(static_cast<unsigned>((n + 255) / 256), a.n), 256, 0, st>>>(
      g.fwd, g.rev, g.factor, h0, dht, one, s.B * s.Hv, s.Hv, s.T, p.segments, p.seg, a.cu);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_chunk_fwd(const LinShape& s, const LinPlan& p, const LinFwdArgs& args, char* ws,
                                hipStream_t st) {
  LinChains a = lin_forward_chains(s, args);
  const LinSegs g = lin_segs(p, false, ws);
  a.segments = p.segments, a.seg = p.seg;
  if (p.segments > 1) {
    LinChains pre = a;
    pre.c[0].s_out = g.fwd;
    if (hipError_t e = segment_states(s, p, g, pre, args.h0, nullptr, st); e != hipSuccess) return e;
    a.c[0].seg_in = g.fwd;
  }
  ProfScope prof("linear_chunks", st);
  return by_type(s.io_bf16, s.Dk, [&](auto op, auto d1) {
    using OP = decltype(op);
    constexpr int D1P = decltype(d1)::value;
    return s.out_bf16 ? run_chunks<OP, D1P, Job<OP::NARROW, false, false>>(a, st)
                      : run_chunks<OP, D1P, Job<OP::FULL, false, true>>(a, st);
  });
}

hipError_t launch_lin_chunk_bwd(const LinShape& s, const LinPlan& p, const LinBwdArgs& args, const LinBwdParts& parts,
                                char* ws, hipStream_t st) {
  LinChains a = lin_backward_chains(s, args, parts);
  const LinSegs g = lin_segs(p, true, ws);
  a.segments = p.segments, a.seg = p.seg;
  if (p.segments > 1) {
    // H forward from (k, v), dS backward from (q, dO), both as [Dk][Dv]
    const LinFwdArgs fwd{args.q, args.k, args.v, args.g, nullptr, nullptr, g.fwd, args.cu};
    LinChains pre = lin_forward_chains(s, fwd);
    pre.n = 2;
    pre.c[1] = a.c[2];
    pre.c[1].s_out = g.rev;
    if (hipError_t e = segment_states(s, p, g, pre, args.h0, args.dht, st); e != hipSuccess) return e;
    a.c[0].seg_in = g.fwd, a.c[0].seg_dot = g.rev;
    a.c[1].seg_in = a.c[2].seg_in = g.rev;
  }
  a.c[0].key = a.c[1].key = 1;
  {
    ProfScope prof("linear_chunks_vjp", st);
    // summed over heads: one launch for each of a key head's value heads, in
    // fp32 rows of the workspace until the last, which dv joins
    a.sum = p.sum;
    const int group = a.group;
    if (p.sum)
      for (int i = 0; i < 2; ++i) {
        a.c[i].out = a.c[i].sum = i ? parts.pdk : parts.pdq;
        a.c[i].og = group;
        a.c[i].out_partial = 1;
      }
    for (a.head = p.sum ? 0 : group - 1; a.head < group; ++a.head) {
      const bool last = a.head + 1 == group;
      a.n = last ? 3 : 2;
      if (p.sum && last) {
        a.c[0].out = args.dq, a.c[1].out = args.dk;
        a.c[0].out_partial = a.c[1].out_partial = 0;
      }
      const bool ex = args.dg != nullptr, add = p.sum && a.head > 0, part = s.Hv != s.Hk && !(p.sum && last);
      const hipError_t e = by_type(s.io_bf16, std::max(s.Dk, s.Dv), [&](auto op, auto d1) {
        using OP = decltype(op);
        constexpr int D1P = decltype(d1)::value;
        return s.out_bf16 ? run_vjp<OP, D1P, false>(a, ex, add, part, st)
                          : run_vjp<OP, D1P, true>(a, ex, add, part, st);
      });
      if (e != hipSuccess) return e;
    }
  }
  // by rows, chunks of 32 tokens leave e in two parts
  const bool cols = s.io_bf16 && (!s.out_bf16 || args.dg), short_chunk = !s.io_bf16 || max_d1(a) > 128;
  const int es = lin_slices(s.Dk) * (short_chunk && !cols ? 2 : 1);
  return launch_lin_bwd_tail(s, args, parts, p.sum, es, 4 * lin_slices(s.Dk), p.segments, p.seg, st);
}

}  // namespace gdr
