// Causal attention over whole sequences with a sliding window and first tokens
// that stay visible, and its VJP.  Per query head, S = scale Q K^T over the pairs
// that are visible, in one pass over the keys:
//     O = sum_j e^{S_ij - m_i} v_j / l_i,   lse_i = m_i + log l_i,
// m the running maximum, O rescaled when it grows.  VJP, with P = e^{S - lse}
// and delta_i = dO_i . O_i:
//     dV = P^T dO,   dS = P o (dO V^T - delta),   dQ = scale dS K,   dK = scale dS^T Q.
//
// All three kernels have one shape.  A wave holds 32 rows of one side as operands
// in its registers (queries; in the dK, dV kernel keys), its workgroup's four
// waves walk tiles of the other side, which go through LDS once for all of them.
// Products of 32 x 32: scores come out as (walked row x held row), a lane holding
// 16 values of one held row, in the order of the next product's summed index, so
// P and dS are operands without a move.  Softmax statistics then need one
// exchange between the wave's halves.  LDS tiles are read by rows (16 bytes a
// lane) and, where they are summed over, by columns (transposing reads); their
// 16-byte units are permuted so that both kinds spread over the banks.
//
// dQ and (dK, dV) are formed by two kernels, each in a fixed order without atomics.
// dK and dV add up over the query heads that share a key head and over the queries.
// How many there are differs by tile (causality, a window, first tokens that every
// query sees) and few tiles do not fill the card, so this work is not cut by tiles:
// it is one list of steps (a tile of queries of one head against a tile of keys), cut
// into equal shares, one for each workgroup that the card holds; a key tile that lies
// in two shares or more is joined by a third launch.  By tiles, with the first ones cut
// apart, the training step below took 1.42 ms instead of 1.31.
//
// Precision.  bf16 inputs are operands as they are; P and dS enter as two bf16
// operands (16 bits) for outputs in bf16 and as three for outputs in fp32: one is
// as coarse as the output itself.  fp32 inputs use fp32 products.
//
// Bound.  The matrix cores and the vector instructions beside them: of S, e^S and its
// two operands a wave issues 5.7-8.7 vector instructions for each product of 32 x 32 x
// 16, which takes as long as 8 of them, and a wave has no other one's to fill the gaps
// (one on a SIMD in the VJP, two in the forward: 18-29 % of a wave's time it waits for
// its turn to issue, 31-50 % for LDS or a barrier, there also for waves whose rows a
// tile's mask leaves; no bank conflicts).  bf16, 32 query and
// 8 key heads of 128, us (a graph of calls): forward, 4 x 4096 tokens, all earlier ones
// visible, 835 (658 TFLOP/s of 4 D a pair; its operands make 1.5 times that: 990); the
// training step of 2 x 4096 tokens under a window of 1024 with 4 sinks 1254 (of a trace's
// 1346 the forward has 234, dQ 477, dK and dV 613, joins 22).  A library product of 8192
// x 8192 x 8192 reaches 1287 TFLOP/s on this card.  Steps that got there: buffers in
// scalar registers, not lane by lane (dK, dV 836 -> 698 us), shares instead of tiles (->
// 639), two products in turn that do not wait for each other (712 -> 578 with pairs
// converted together), masks in a branch of their own, addresses formed once.  Set aside:
// two waves for dV and dK at 128 channels (more products, the same time), the next rows
// read before the products (1 %), one code path for each LDS buffer (spills), the
// compiler's interleaving hints (2 % more).

#include <algorithm>
#include <type_traits>

#include "gdr_attn.h"
#include "gdr_device.h"

namespace gdr {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kHeld = 32, kWaves = 4, kBlock = kHeld * kWaves;  // held rows of a wave, of a workgroup

__device__ __forceinline__ int lane_id() { return threadIdx.x & 63; }

// What is the same in a whole wave, kept in scalar registers: the compiler does not
// see it through 64-bit arithmetic, and would load from a buffer lane by lane.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = uniform(static_cast<int>(x)), hi = uniform(static_cast<int>(x >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ int wave_id() { return uniform(static_cast<int>(threadIdx.x >> 6)); }

// Element types: PER elements in 16 bytes, TILE rows walked at a time.
template <typename T> struct El;
template <> struct El<bf16_t> {
  static constexpr int PER = 8, TILE = 64;
};
template <> struct El<float> {
  static constexpr int PER = 4, TILE = 32;
};

// Tiles of ROWS x DP of two tensors in LDS, BUFS times.  Unit u (16 bytes) of a row
// lies at u ^ mix(row): rows read together by a wave's 16-lane groups fall on
// different banks.
template <typename T_, int DP_, int ROWS_ = El<T_>::TILE, int BUFS_ = 2> struct Tile {
  using T = T_;
  static constexpr int DP = DP_, ROWS = ROWS_, BUFS = BUFS_;
  static constexpr int PER = El<T>::PER, UNITS = DP / PER, KF = UNITS / 2, PITCH = UNITS * 16;
  static constexpr int BYTES = ROWS * PITCH, PAIR = 2 * BYTES, LOADS = ROWS * UNITS / 256;
  static __device__ __forceinline__ int mix(int row) {
    return UNITS == 8 ? ((row >> 1 & 1) << 2 | (row >> 2 & 3)) : ((row & 3) << 2 | (row >> 2 & 3));
  }
  static __device__ __forceinline__ int at(int row, int unit) { return row * PITCH + ((unit ^ mix(row)) << 4); }
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t kNowhere = 0x7fffffffu;  // an offset past any buffer's end

// Rows of a tensor [.., rows, heads, D] for one sequence and head.
struct Rows {
  const char* base;     // the sequence's first row, the head's first channel
  uint32_t pitch;       // bytes between rows
  int n, bytes;         // rows of the sequence; bytes of a row
  // Rows row0 .. row0 + count - 1 as a buffer: what lies past the sequence's end
  // reads as zero.
  __device__ __forceinline__ rsrc_t buffer(int row0, int count) const {
    const int left = max(0, min(n - row0, count));
    const int64_t at = uniform(reinterpret_cast<int64_t>(base) + static_cast<int64_t>(min(row0, n)) * pitch);
    const int size = uniform(left ? (left - 1) * static_cast<int>(pitch) + bytes : 0);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), 0, size, 0x00020000);
  }
};
template <typename T>
__device__ __forceinline__ Rows rows_of(const void* p, int64_t start, int n, int64_t row, int head, int D) {
  return {static_cast<const char*>(p) + (start * row + static_cast<int64_t>(head) * D) * sizeof(T),
          static_cast<uint32_t>(row * sizeof(T)), n, D * static_cast<int>(sizeof(T))};
}
__device__ __forceinline__ u32x4 load16(rsrc_t b, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(at), 0, 0));
}

// A tile on its way to LDS through registers; the offsets are formed once.
template <typename L> struct Staged {
  u32x4 x[L::LOADS];
  uint32_t from[L::LOADS];
  __device__ __forceinline__ void init(const Rows& r) {
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i) {
      const int idx = threadIdx.x + 256 * i, row = idx / L::UNITS, u = idx % L::UNITS;
      from[i] = u * 16 < r.bytes ? row * r.pitch + u * 16 : kNowhere;
    }
  }
  __device__ __forceinline__ void load(const Rows& r, int row0) {
    const rsrc_t b = r.buffer(row0, L::ROWS);
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i) x[i] = load16(b, from[i]);
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i) {
      const int idx = threadIdx.x + 256 * i;
      *reinterpret_cast<u32x4*>(lds + L::at(idx / L::UNITS, idx % L::UNITS)) = x[i];
    }
  }
};

// A wave's held rows as the second operand: lane (row lane % 32, units 2 i + lane / 32).
template <typename L>
__device__ __forceinline__ void load_held(const Rows& r, int row0, u32x4 (&f)[L::KF]) {
  const rsrc_t b = r.buffer(row0, kHeld);
  const int row = lane_id() & 31, h = lane_id() >> 5;
#pragma unroll
  for (int i = 0; i < L::KF; ++i)
    f[i] = load16(b, (2 * i + h) * 16 < r.bytes ? row * r.pitch + (2 * i + h) * 16 : kNowhere);
}

template <typename T>
__device__ __forceinline__ f32x16 mma(u32x4 x, u32x4 y, f32x16 c) {
  if constexpr (sizeof(T) == 2) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0,
                                                   0, 0);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(x[e]), __uint_as_float(y[e]), c, 0, 0, 0);
    return c;
  }
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// A lane's places in a tile, formed once: of by_rows' units, and of by_columns' runs
// of 4 channels (rows 4 h .. + 3, and 8 rows on).  Units 16 apart lie 256 bytes
// apart, rows 16 apart 16 rows: constants of the reads.  flip() goes to the other
// buffer.
template <typename L> struct Lane {
  static constexpr int NR = L::KF < 8 ? L::KF : 8, NC = L::PER == 4 ? 0 : L::DP / 32 < 4 ? L::DP / 32 : 4;
  int row[NR], col[NC ? NC : 1][2], one;
  __device__ __forceinline__ Lane(int row0) {
    const int lane = lane_id(), h = lane >> 5, q = lane & 15, side = lane >> 4 & 1;
    one = row0 * L::PITCH;
#pragma unroll
    for (int i = 0; i < NR; ++i) row[i] = one + L::at(lane & 31, 2 * i + h);
#pragma unroll
    for (int t = 0; t < NC; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        col[t][k] = one + L::at(4 * h + (q >> 2) + 8 * k, 4 * t + 2 * side + (q >> 1 & 1)) + (q & 1) * 8;
  }
  __device__ __forceinline__ void flip() {
    if constexpr (L::BUFS == 1) return;
    one ^= L::PAIR;
#pragma unroll
    for (int i = 0; i < NR; ++i) row[i] ^= L::PAIR;
#pragma unroll
    for (int t = 0; t < NC; ++t) col[t][0] ^= L::PAIR, col[t][1] ^= L::PAIR;
  }
};

// (rows row0 .. + 31 of the tile) x (held rows): lane (held row lane % 32) holds
// tile rows row0 + 8 (i / 4) + 4 (lane / 32) + i % 4.
template <typename L>
__device__ __forceinline__ u32x4 unit(const Lane<L>& at, const char* lds, int row0, int i) {
  return *reinterpret_cast<const u32x4*>(lds + at.row[i & 7] + (row0 * L::PITCH + (i >> 3) * 256));
}
template <typename L>
__device__ __forceinline__ f32x16 by_rows(const Lane<L>& at, const char* lds, int row0, const u32x4 (&held)[L::KF]) {
  f32x16 c = zero16();
#pragma unroll
  for (int i = 0; i < L::KF; ++i) c = mma<typename L::T>(unit<L>(at, lds, row0, i), held[i], c);
  return c;
}
// Two such products in turn: each waits for its own last one, not for the other's.
template <typename L>
__device__ __forceinline__ void by_rows2(const Lane<L>& at, const char* lds0, const char* lds1, int row0, int row1,
                                         const u32x4 (&held0)[L::KF], const u32x4 (&held1)[L::KF], f32x16& c0,
                                         f32x16& c1) {
  c0 = zero16(), c1 = zero16();
#pragma unroll
  for (int i = 0; i < L::KF; ++i) {
    c0 = mma<typename L::T>(unit<L>(at, lds0, row0, i), held0[i], c0);
    c1 = mma<typename L::T>(unit<L>(at, lds1, row1, i), held1[i], c1);
  }
}
// Of element i, the tile row less 4 (lane / 32).
__device__ constexpr int walked(int i) { return 8 * (i >> 2) + (i & 3); }

// NP bf16 parts of eight values, most significant first; converted in pairs.
template <int NP>
__device__ __forceinline__ void split(const float* p, bf16x8 (&out)[NP]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 w[NP];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x2 r{p[2 * i], p[2 * i + 1]};
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      w[k][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(r, bf16x2));
      r[0] -= __uint_as_float(w[k][i] << 16);
      r[1] -= __uint_as_float(w[k][i] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int k = 0; k < NP; ++k) out[k] = __builtin_bit_cast(bf16x8, w[k]);
}

// acc[t] += (channels 32 t .. + 31 of tile rows row0 .. + 31)^T x p, p as by_rows
// gives it: lane (held row) then has channels 32 t + 4 (lane / 32) + walked(i).  With
// MORE, more += the same of y, as one bf16 operand.  half: the bytes from a tile's row
// to the one 16 rows on.
template <typename L, int NP, bool MORE = false>
__device__ __forceinline__ void by_columns(f32x16 (&acc)[L::DP / 32], const Lane<L>& at, const char* lds, int row0,
                                           const float (&p)[16], f32x16* more = nullptr, const float* y = nullptr,
                                           int half = 16 * L::PITCH) {
  constexpr int NT = L::DP / 32;
  if constexpr (L::PER == 8) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 f[NP], g[1];
      split<NP>(p + 8 * k, f);
      if constexpr (MORE) split<1>(y + 8 * k, g);
      bf16x8 x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const char* from = lds + (row0 * L::PITCH + k * half + (t >> 2) * 256);
        const bf16x4 a = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(from + at.col[t & 3][0])));
        const bf16x4 b = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(from + at.col[t & 3][1])));
        x[t] = bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      }
      // a sum's products one after another would wait for each other
#pragma unroll
      for (int n = NP - 1; n >= 0; --n)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[t], f[n], acc[t], 0, 0, 0);
      if constexpr (MORE)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          more[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[t], g[0], more[t], 0, 0, 0);
    }
  } else {
    const int d = lane_id() & 31, h = lane_id() >> 5;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = walked(i) + 4 * h;
        const float x = *reinterpret_cast<const float*>(
            lds + at.one + (row0 + (r & 15)) * L::PITCH + (i >> 3) * half +
            (((8 * t + (d >> 2)) ^ L::mix(r)) << 4) + (d & 3) * 4);
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, p[i], acc[t], 0, 0, 0);
        if constexpr (MORE) more[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, y[i], more[t], 0, 0, 0);
      }
  }
}

// Four results; bf16 by the conversion instruction (to nearest, ties to even).
template <typename TO>
__device__ __forceinline__ void store4(TO* at, const float (&x)[4]) {
  if constexpr (sizeof(TO) == 2) {
    *reinterpret_cast<bf16x4*>(at) = bf16x4{static_cast<__bf16>(x[0]), static_cast<__bf16>(x[1]),
                                            static_cast<__bf16>(x[2]), static_cast<__bf16>(x[3])};
  } else {
    st4<TO>(at, x);
  }
}

// A wave's held rows, channels 32 t + walked(i) each, times f, to rows of `out`.
template <typename TO, int NT>
__device__ __forceinline__ void store_held(TO* out, int64_t pitch, const f32x16 (&acc)[NT], float f, int D) {
  TO* at = out + static_cast<int64_t>(lane_id() & 31) * pitch + 4 * (lane_id() >> 5);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (32 * t + 8 * b + 4 * (lane_id() >> 5) >= D) continue;
      const float x[4] = {acc[t][4 * b] * f, acc[t][4 * b + 1] * f, acc[t][4 * b + 2] * f, acc[t][4 * b + 3] * f};
      store4<TO>(at + 32 * t + 8 * b, x);
    }
}

// A sequence of the batch: its first row and its length.
struct Span {
  int64_t start;
  int n;
};
__device__ __forceinline__ Span span(const AttnArgs& a, int64_t b) {
  if (!a.cu) return {b * a.T, static_cast<int>(a.T)};
  const int64_t lo = a.cu[b];
  return {lo, static_cast<int>(max(int64_t(0), min(a.cu[b + 1] - lo, a.T)))};
}

// Visible: j <= i and (no window, or i - j < window, or j < sinks).
struct Mask {
  int window, sinks;
  __device__ __forceinline__ Mask(const AttnArgs& a) : window(static_cast<int>(a.window)), sinks(static_cast<int>(a.sinks)) {}
  __device__ __forceinline__ bool sees(int i, int j) const {
    return j <= i && (window == 0 || i - j < window || j < sinks);
  }
  // all pairs of i0 .. i1 and j0 .. j1; none of them
  __device__ __forceinline__ bool all(int i0, int i1, int j0, int j1) const {
    return j1 <= i0 && (window == 0 || i1 - j0 < window || j1 < sinks);
  }
  __device__ __forceinline__ bool none(int i0, int i1, int j0, int j1) const {
    return j0 > i1 || (window != 0 && i0 - j1 >= window && j0 >= sinks);
  }
};
// Keeps what follows in a branch: the compiler would mask every tile, not the few
// that need it.
__device__ __forceinline__ void rarely() { asm volatile(""); }

// Key tiles that queries q0 .. q1 see, as a list: sinks, then the window.
struct KeyTiles {
  int head, skip, count;
  __device__ __forceinline__ KeyTiles(const Mask& m, int q0, int q1, int tile) {
    const int first = m.window == 0 ? 0 : max(0, q0 - m.window + 1) / tile;
    head = m.window == 0 ? 0 : min((m.sinks + tile - 1) / tile, first);
    skip = first - head;
    count = q1 / tile + 1 - skip;
  }
  __device__ __forceinline__ int operator[](int i) const { return i < head ? i : i + skip; }
};

// The VJP's kernels have two sums for their held rows (dV and dK; dS K and P K).
// One wave forms both, for each of four blocks of 32 rows; where its registers are far
// from holding them (256 channels in bf16) two waves do, one sum each, for each of two
// blocks.  That costs the scores twice, but 2 x 2048 tokens of 16 heads of 256 take 0.98
// ms instead of 1.90, of which spilled registers were the most.  At 128 channels two waves
// for each block, all eight on a compute unit, took the same time (1.24 ms for the
// training step of 2 x 4096 tokens), and fp32 up to a quarter more.
//
// What still spills, registers of a lane.  bf16 at 256 channels: dK, dV 48-52, the narrow
// forward 44, the narrow dQ with fp32 outputs 192.  fp32 at 128: the wide forward 30, dK,
// dV 12, dQ with bf16 outputs 27-166.  fp32 at 256 (where one wave forms both sums): the
// forward 114, dQ 223-341, dK, dV 494.
template <typename T, int DP> constexpr bool kApart = sizeof(T) == 2 && DP > 128;
template <typename T, int DP> constexpr int kBlocks = kApart<T, DP> ? 2 : 4;
// Workgroups of these kernels on a compute unit.
template <typename T, int DP> constexpr int kResident = sizeof(T) == 2 && DP <= 64 ? 2 : 1;
constexpr int kBoth = 0, kFirst = 1, kSecond = 2;  // what a wave forms

// Rows of a tile of which a wave's mask leaves nothing: their weights are 0, but 0 times
// an Inf or NaN in them is NaN, so they may not enter a product.  The VJP's kernels
// branch around such 32 rows (0: no zeros), or, where a branch makes the compiler move
// or spill sums, take zeros in their place, which lie behind the tiles: 32 rows of
// them, or 16 that are read twice where LDS holds no more.  us, neither : branch : zeros.
// dK, dV: fp32, 2 x 1024 tokens of 32 heads of 128 386 : 502 : 408; 700 of 16 heads of
// 256 424 : 517 : 340; 2 x 1024 of 16 heads of 64 112 : 113 : 125; bf16, 2 x 2048 of 16
// heads of 256 460 : 444 : 492 (in fp32 out 452 : 477 : 472).  dQ, at the first two
// 371 : 354 : 464, 457 : 554 : 494, bf16, 777 tokens of 8 heads of 80 23.7 : 26.5 : 24.1.
template <typename T, int DP, bool WIDE>
constexpr int kZerosDq = sizeof(T) == 2 ? (WIDE ? 0 : 16) : DP > 128 ? 16 : 0;
template <typename T, int DP>
constexpr int kZerosDkv = sizeof(T) == 2 || DP <= 64 ? 0 : DP <= 128 ? 32 : 16;
template <typename L, int ZEROS> __device__ __forceinline__ void clear_zeros(char* lds) {
  for (int i = threadIdx.x * 16; i < ZEROS * L::PITCH; i += 256 * 16)
    *reinterpret_cast<u32x4*>(lds + L::BUFS * L::PAIR + i) = u32x4{0, 0, 0, 0};
}
// Where by_columns finds rows row0 .. of a tensor's tile, or with `none` the zeros.
template <typename L, int ZEROS>
__device__ __forceinline__ const char* rows_or_zeros(const Lane<L>& at, const char* lds, int row0, int tensor, bool none) {
  return ZEROS && none ? lds + (L::BUFS * L::PAIR - at.one - row0 * L::PITCH) : lds + tensor;
}
template <typename L, int ZEROS> __device__ __forceinline__ int half_of(bool none) {
  return ZEROS == 16 && none ? 0 : 16 * L::PITCH;
}

// The layout of the kernels that hold queries.  WIDE: each of N waves holds 32
// queries of its own and walks all rows of a tile.  Otherwise all hold the same 32, and
// each takes 32 rows of a tile of 32 N, for grids that do not fill the card: N times
// the workgroups, each an N-th as long, joined at its end.
template <typename T, int DP, int N, bool WIDE>
using QTile = Tile<T, DP, WIDE ? El<T>::TILE : 32 * N,
                   WIDE || 128 * N * DP * sizeof(T) <= (128 << 10) ? 2 : 1>;

// What the waves of a workgroup hold of the same queries, added: wave w is left with
// the sums of channels 32 t, t = w, w + N, ..
template <int N, int NT>
__device__ __forceinline__ void add_waves(f32x16 (&acc)[NT], int wave, char* lds) {
  float* at = reinterpret_cast<float*>(lds) + lane_id();
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) at[((wave * NT + t) * 16 + i) * 64] = acc[t][i];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t % N != wave) continue;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = at[(t * 16 + i) * 64];
#pragma unroll
      for (int w = 1; w < N; ++w) x += at[((w * NT + t) * 16 + i) * 64];
      acc[t][i] = x;
    }
  }
}
template <typename TO, int N, int NT>
__device__ __forceinline__ void store_own(TO* out, int64_t pitch, const f32x16 (&acc)[NT], int wave, float f, int D) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
    if (t % N == wave) {
      const f32x16 one[1] = {acc[t]};
      store_held<TO, 1>(out + 32 * t, pitch, one, f, D - 32 * t);
    }
}

template <typename T, typename TO, int DP, int NP, bool WIDE>
__global__ __launch_bounds__(256, WIDE && DP <= 128 ? 2 : 1) void attn_fwd_kernel(AttnArgs a) {
  using L = QTile<T, DP, kWaves, WIDE>;
  constexpr int NT = DP / 32, BLOCK = WIDE ? kBlock : kHeld, SUB = WIDE ? L::ROWS / 32 : 1;
  __shared__ __align__(16) char lds[L::BUFS * L::PAIR];
  __shared__ float stat[WIDE ? 1 : kWaves][2][32];
  const int h = blockIdx.x, kh = h / (a.Hq / a.Hk), lane = lane_id(), wave = wave_id();
  const Span s = span(a, blockIdx.z);
  const int block0 = static_cast<int>(gridDim.y - 1 - blockIdx.y) * BLOCK;  // long rows first
  if (block0 >= s.n) return;
  const Mask mask(a);
  const KeyTiles tiles(mask, block0, min(block0 + BLOCK, s.n) - 1, L::ROWS);
  const Rows kr = rows_of<T>(a.k, s.start, s.n, a.k_row, kh, a.D), vr = rows_of<T>(a.v, s.start, s.n, a.v_row, kh, a.D);
  const int q0 = block0 + (WIDE ? wave * kHeld : 0), q1 = q0 + kHeld - 1, qi = q0 + (lane & 31);
  const int mine0 = WIDE ? 0 : 32 * wave;  // the wave's rows of a tile
  Staged<L> ks, vs;
  ks.init(kr), vs.init(vr);
  ks.load(kr, tiles[0] * L::ROWS), vs.load(vr, tiles[0] * L::ROWS);
  u32x4 qf[L::KF];
  load_held<L>(rows_of<T>(a.q, s.start, s.n, a.q_row, h, a.D), q0, qf);
  f32x16 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = zero16();
  float m = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;
  const int count = uniform(tiles.count);
  Lane<L> at(mine0);
  int fill = 0;  // where the next tile goes
  ks.store(lds), vs.store(lds + L::BYTES);
  for (int it = 0; it < count; ++it) {
    __syncthreads();
    if (it + 1 < count) ks.load(kr, tiles[it + 1] * L::ROWS), vs.load(vr, tiles[it + 1] * L::ROWS);
    if constexpr (L::BUFS == 2) fill ^= L::PAIR;
    const int j0 = tiles[it] * L::ROWS + mine0, j1 = j0 + 32 * SUB - 1;
    if (!mask.none(q0, q1, j0, j1)) {
      float x[SUB][16];
      if constexpr (SUB == 2) {
        f32x16 c, d;
        by_rows2<L>(at, lds, lds, 0, 32, qf, qf, c, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[0][i] = c[i], x[1][i] = d[i];
      } else {
        const f32x16 c = by_rows<L>(at, lds, 0, qf);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[0][i] = c[i];
      }
      if (!mask.all(q0, q1, j0, j1)) {
        rarely();
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!mask.sees(qi, j0 + 4 * (lane >> 5) + 32 * u + walked(i))) x[u][i] = -INFINITY;
      }
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[u][i]);
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      if (__any(top > m)) {
        top = fmaxf(top, m);
        const float f = m == -INFINITY ? 0.f : exp2f((m - top) * c2);
        l *= f;
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] *= f;
        m = top;
      }
      const float mc = m == -INFINITY ? 0.f : m * c2;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[u][i] = __builtin_amdgcn_exp2f(fmaf(x[u][i], c2, -mc));
          l += x[u][i];
        }
        by_columns<L, NP>(acc, at, lds + L::BYTES, 32 * u, x[u]);
      }
    }
    if constexpr (L::BUFS == 1) __syncthreads();
    if (it + 1 < count) ks.store(lds + fill), vs.store(lds + fill + L::BYTES);
    at.flip();
  }
  l += __shfl_xor(l, 32, 64);
  const int64_t pitch = static_cast<int64_t>(a.Hq) * a.D;
  TO* out = static_cast<TO*>(a.o) + (s.start + q0) * pitch + static_cast<int64_t>(h) * a.D;
  if constexpr (!WIDE) {
    if (lane < 32) stat[wave][0][lane] = m, stat[wave][1][lane] = l;
    __syncthreads();  // also: the tiles are read
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[w][0][lane & 31]);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = stat[w][0][lane & 31];
      l += stat[w][1][lane & 31] * (mw == -INFINITY ? 0.f : exp2f((mw - top) * c2));
    }
    const float f = m == -INFINITY ? 0.f : exp2f((m - top) * c2);
    m = top;
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] *= f;
    add_waves<kWaves>(acc, wave, lds);
    if (qi >= s.n) return;
    store_own<TO, kWaves>(out, pitch, acc, wave, 1.f / l, a.D);
    if (wave > 0) return;
  } else {
    if (qi >= s.n) return;
    store_held<TO, NT>(out, pitch, acc, 1.f / l, a.D);
  }
  if (lane < 32) a.lse[(s.start + qi) * a.Hq + h] = fmaf(m, a.scale, log2f(l) * kLn2);
}

// dQ, and delta into the workspace (the next kernel reads it).
//
// delta = dO . O with an O rounded to bf16 is off by 2^-9 of its terms, more than
// dS itself where one key has most of a row's weight.  So with a bf16 O the sum of
// dS over the keys, which is 0 for the right delta, is what delta is off by (e):
// dQ has e (P K) taken off (K^T is in registers for dS; one bf16 operand for P is
// enough, as e is small), and the delta that is passed on has e added.
template <typename T, typename TO, int DP, bool WIDE> struct Dq {
  static constexpr bool FIX = sizeof(TO) == 2, APART = FIX && kApart<T, DP>;
  static constexpr int N = APART ? 2 : 4, BLOCK = kHeld * (WIDE ? N : 1);
  using L = QTile<T, DP, N, WIDE>;
};
template <typename T, typename TO, int DP, int NP, bool WIDE>
__global__ __launch_bounds__(256, (kResident<T, DP>)) void attn_dq_kernel(AttnArgs a) {
  using C = Dq<T, TO, DP, WIDE>;
  using L = typename C::L;
  constexpr int NT = DP / 32, N = C::N, SUB = WIDE ? L::ROWS / 32 : 1, ZEROS = kZerosDq<T, DP, WIDE>;
  __shared__ __align__(16) char lds[L::BUFS * L::PAIR + ZEROS * L::PITCH];
  __shared__ float stat[N][32];
  clear_zeros<L, ZEROS>(lds);
  const int h = blockIdx.x, kh = h / (a.Hq / a.Hk), lane = lane_id();
  const int wave = wave_id() % N;
  const Span s = span(a, blockIdx.z);
  const int block0 = static_cast<int>(gridDim.y - 1 - blockIdx.y) * C::BLOCK;
  if (block0 >= s.n) return;
  const Mask mask(a);
  const KeyTiles tiles(mask, block0, min(block0 + C::BLOCK, s.n) - 1, L::ROWS);
  const Rows kr = rows_of<T>(a.k, s.start, s.n, a.k_row, kh, a.D), vr = rows_of<T>(a.v, s.start, s.n, a.v_row, kh, a.D);
  const int q0 = block0 + (WIDE ? wave * kHeld : 0), q1 = q0 + kHeld - 1, qi = q0 + (lane & 31);
  const int mine0 = WIDE ? 0 : 32 * wave;
  const int64_t pitch = static_cast<int64_t>(a.Hq) * a.D;
  Staged<L> ks, vs;
  ks.init(kr), vs.init(vr);
  ks.load(kr, tiles[0] * L::ROWS), vs.load(vr, tiles[0] * L::ROWS);
  float lse2 = 0.f;
  if (qi < s.n) lse2 = a.lse_in[(s.start + qi) * a.Hq + h] * kLog2e;
  const float c2 = a.scale * kLog2e;
  const int count = uniform(tiles.count);
  TO* out = static_cast<TO*>(a.dq) + (s.start + q0) * pitch + static_cast<int64_t>(h) * a.D;
  // e (P K) on its way to the wave that has dS K
  float* const meet = reinterpret_cast<float*>(lds) + wave * (NT * 16 * 64) + lane;
  // all tiles of a wave, which forms dS K, P K (the second sum) or both
  auto walk = [&](auto what) {
    constexpr int WHAT = decltype(what)::value;
    constexpr bool SECOND = WHAT == kSecond, PK = C::FIX && WHAT == kBoth;
    u32x4 qf[L::KF], df[SECOND ? 1 : L::KF];
    load_held<L>(rows_of<T>(a.q, s.start, s.n, a.q_row, h, a.D), q0, qf);
    float delta = 0.f;
    if constexpr (!SECOND) {
      load_held<L>(rows_of<T>(a.dout, s.start, s.n, pitch, h, a.D), q0, df);
      if (qi < s.n) {
        const TO* o = static_cast<const TO*>(a.out) + (s.start + qi) * pitch + static_cast<int64_t>(h) * a.D;
#pragma unroll
        for (int i = 0; i < L::KF; ++i) {
          const int d = (2 * i + (lane >> 5)) * L::PER;
          if (d >= a.D) continue;
#pragma unroll
          for (int e = 0; e < L::PER; e += 4) {
            float y[4];
            ld4<TO>(o + d + e, y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x = sizeof(T) == 4 ? __uint_as_float(df[i][k])
                              : k & 1        ? __uint_as_float(df[i][(e + k) / 2] & 0xffff0000u)
                                             : __uint_as_float(df[i][(e + k) / 2] << 16);
              delta += x * y[k];
            }
          }
        }
      }
      delta += __shfl_xor(delta, 32, 64);
    }
    f32x16 acc[NT], pk[PK ? NT : 1];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      acc[t] = zero16();
      if constexpr (PK) pk[t] = zero16();
    }
    float off = 0.f;
    Lane<L> at(mine0);
    int fill = 0;
    ks.store(lds), vs.store(lds + L::BYTES);
    for (int it = 0; it < count; ++it) {
      __syncthreads();
      if (it + 1 < count) ks.load(kr, tiles[it + 1] * L::ROWS), vs.load(vr, tiles[it + 1] * L::ROWS);
      if constexpr (L::BUFS == 2) fill ^= L::PAIR;
      const int j0 = tiles[it] * L::ROWS + mine0;
      const bool all = mask.all(q0, q1, j0, j0 + 32 * SUB - 1);
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const bool none = mask.none(q0, q1, j0 + 32 * u, j0 + 32 * u + 31);
        if (ZEROS == 0 && none) continue;
        f32x16 c, dp;
        float x[16], p[16];
        if constexpr (SECOND) {
          c = by_rows<L>(at, lds, 32 * u, qf);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __builtin_amdgcn_exp2f(fmaf(c[i], c2, -lse2));
        } else {
          by_rows2<L>(at, lds, lds + L::BYTES, 32 * u, 32 * u, qf, df, c, dp);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(c[i], c2, -lse2));
            x[i] = p[i] * (dp[i] - delta);
          }
        }
        if (!all) {
          rarely();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!mask.sees(qi, j0 + 4 * (lane >> 5) + 32 * u + walked(i))) x[i] = 0.f, p[i] = 0.f;
        }
        if constexpr (C::FIX && !SECOND)
#pragma unroll
          for (int i = 0; i < 16; ++i) off += x[i];
        by_columns<L, SECOND ? 1 : NP, PK>(acc, at, rows_or_zeros<L, ZEROS>(at, lds, 32 * u, 0, none), 32 * u, x, pk, p,
                                           half_of<L, ZEROS>(none));
      }
      if constexpr (L::BUFS == 1) __syncthreads();
      if (it + 1 < count) ks.store(lds + fill), vs.store(lds + fill + L::BYTES);
      at.flip();
    }
    if constexpr (C::FIX) {
      if constexpr (!SECOND) {
        off += __shfl_xor(off, 32, 64);
        if (lane < 32) stat[wave][lane] = off;
      }
      __syncthreads();  // also: the tiles are read
      off = stat[WIDE ? wave : 0][lane & 31];
      if constexpr (!WIDE)
#pragma unroll
        for (int w = 1; w < N; ++w) off += stat[w][lane & 31];
      delta += off;
      if constexpr (PK) {
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] -= off * pk[t];
      } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if constexpr (SECOND) meet[(t * 16 + i) * 64] = off * acc[t][i];
        __syncthreads();
        if constexpr (!SECOND)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[t][i] -= meet[(t * 16 + i) * 64];
      }
    }
    if constexpr (!WIDE) {
      __syncthreads();
      if constexpr (SECOND) {
        __syncthreads();  // add_waves has one
        return;
      }
      add_waves<N>(acc, wave, lds);
      if (qi >= s.n) return;
      store_own<TO, N>(out, pitch, acc, wave, a.scale, a.D);
      if (wave > 0) return;
    } else {
      if (SECOND || qi >= s.n) return;
      store_held<TO, NT>(out, pitch, acc, a.scale, a.D);
    }
    if (lane < 32) reinterpret_cast<float*>(a.ws)[(s.start + qi) * a.Hq + h] = delta;
  };
  if constexpr (C::APART) {
    if (wave_id() < N) walk(std::integral_constant<int, kFirst>{});
    else walk(std::integral_constant<int, kSecond>{});
  } else {
    walk(std::integral_constant<int, kBoth>{});
  }
}

// The work of dK and dV: steps (a tile of queries of one head, against a tile of
// BLOCK keys), for a sequence and key head key tile by key tile, in each head by
// head.  Key tile t is seen by query tiles from its own on: to the sequence's end
// (no window, or first tokens in it), else `reach` of them.
template <int R, int BLOCK>  // rows of a query tile and of a key tile
struct Steps {
  static constexpr int PER = BLOCK / R;  // query tiles of a key tile's length
  int group, tiles, queries, sinks, reach;
  __host__ __device__ __forceinline__ Steps(int64_t n, int group, int64_t window, int64_t sink)
      : group(group), tiles(static_cast<int>((n + BLOCK - 1) / BLOCK)), queries(static_cast<int>((n + R - 1) / R)),
        sinks(window ? static_cast<int>((sink + BLOCK - 1) / BLOCK) : tiles),
        reach(static_cast<int>((BLOCK - 2 + window) / R + 1)) {
    if (sinks > tiles) sinks = tiles;
  }
  // query tiles that see key tile t
  __host__ __device__ __forceinline__ int seen(int t) const {
    const int all = queries - PER * t;
    return t < sinks || all < reach ? all : reach;
  }
  // steps of the key tiles before t
  __host__ __device__ __forceinline__ int64_t before(int64_t t) const {
    const auto full = [&](int64_t x) { return x * queries - PER * (x * (x - 1) / 2); };
    if (t <= sinks) return group * full(t);
    int64_t cut = queries >= reach ? (queries - reach) / PER + 1 : 0;  // from here on the end is nearer
    cut = cut < sinks ? sinks : cut > t ? t : cut;
    return group * (full(sinks) + (cut - sinks) * reach + full(t) - full(cut));
  }
  // the key tile of a step
  __device__ __forceinline__ int tile_of(int64_t step) const {
    int lo = 0, hi = tiles - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (before(mid) <= step) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// All steps of a batch, cut into one share for each workgroup.
template <int R, int BLOCK>
__device__ __forceinline__ Steps<R, BLOCK> steps_of(const AttnArgs& a, int64_t b) {
  return Steps<R, BLOCK>(span(a, b).n, a.Hq / a.Hk, a.window, a.sinks);
}
template <int R, int BLOCK>
__device__ __forceinline__ int64_t steps_all(const AttnArgs& a, int64_t b) {
  const Steps<R, BLOCK> s = steps_of<R, BLOCK>(a, b);
  return s.before(s.tiles) * a.Hk;
}
__device__ __forceinline__ int64_t shfl64(int64_t x, int lane) {
  const uint32_t lo = __shfl(static_cast<int>(x), lane, 64), hi = __shfl(static_cast<int>(x >> 32), lane, 64);
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}
// Inclusive sums over the lanes.
__device__ __forceinline__ int64_t sums64(int64_t x) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t y = shfl64(x, lane_id() - d < 0 ? 0 : lane_id() - d);
    if (lane_id() >= d) x += y;
  }
  return x;
}
// A step's place: its sequence (B: past the last), key head, key tile, and step in the
// tile.
template <int R, int BLOCK> struct Place {
  int64_t b, step;
  int kh, tile;
  __device__ __forceinline__ Place(const AttnArgs& a, int64_t x) : b(0), step(0), kh(0), tile(0) {
    if (!a.cu) {
      const int64_t each = steps_all<R, BLOCK>(a, 0);
      b = x / each;
      x -= b * each;
    } else {
      for (;; b += 64) {
        if (b >= a.B) {
          b = a.B;
          return;
        }
        const int64_t own = b + lane_id() < a.B ? steps_all<R, BLOCK>(a, b + lane_id()) : 0, upto = sums64(own);
        const uint64_t past = __ballot(upto > x);
        if (past) {
          const int at = __builtin_ctzll(past);
          b += at;
          x -= shfl64(upto - own, at);
          break;
        }
        x -= shfl64(upto, 63);
      }
    }
    const Steps<R, BLOCK> s = steps_of<R, BLOCK>(a, b);
    const int64_t head = s.before(s.tiles);
    kh = static_cast<int>(x / head);
    x -= kh * head;
    tile = s.tile_of(x);
    step = x - s.before(tile);
  }
};
template <int R, int BLOCK>
__device__ __forceinline__ int64_t share_of(const AttnArgs& a, int shares) {
  int64_t all = 0;
  if (!a.cu) {
    all = steps_all<R, BLOCK>(a, 0) * a.B;
  } else {
    for (int64_t b = 0; b < a.B; b += 64) all += shfl64(sums64(b + lane_id() < a.B ? steps_all<R, BLOCK>(a, b + lane_id()) : 0), 63);
  }
  return max(int64_t(1), (all + shares - 1) / shares);
}

// Partial sums of key tiles that several shares have a part of: a share has at most
// two, the tile that it begins in the middle of and the one that it ends in.
struct Parts {
  float *delta, *sums;
};
template <int DP, int BLOCK>
__device__ __forceinline__ float* part_of(const Parts& p, int64_t share, bool end) {
  return p.sums + (2 * share + end) * (2 * BLOCK * DP);
}

template <typename T, typename TO, int DP, int NP>
__global__ __launch_bounds__(256, (kResident<T, DP>)) void attn_dkv_kernel(AttnArgs a, Parts parts) {
  constexpr int N = kBlocks<T, DP>, BLOCK = kHeld * N;
  using L = Tile<T, DP>;
  constexpr int NT = DP / 32, R = L::ROWS, ZEROS = kZerosDkv<T, DP>;
  __shared__ __align__(16) char lds[2 * L::PAIR + ZEROS * L::PITCH];
  __shared__ __align__(16) float stat[2][2][R];
  clear_zeros<L, ZEROS>(lds);
  const int group = a.Hq / a.Hk, lane = lane_id(), wave = wave_id() % N;
  const int64_t share = uniform(share_of<R, BLOCK>(a, gridDim.x));
  Place<R, BLOCK> at(a, share * blockIdx.x);
  const Mask mask(a);
  const float c2 = a.scale * kLog2e;
  const int64_t pitch = static_cast<int64_t>(a.Hq) * a.D, kp = static_cast<int64_t>(a.Hk) * a.D;
  for (int64_t left = share; left > 0;) {
    const int64_t b = uniform(at.b);
    if (b >= a.B) return;
    const Span s{uniform(span(a, b).start), uniform(span(a, b).n)};
    const Steps<R, BLOCK> steps(s.n, group, a.window, a.sinks);
    const int kh = uniform(at.kh), kt = uniform(at.tile), block0 = kt * BLOCK;
    const int per = steps.seen(kt);
    const int64_t total = static_cast<int64_t>(per) * group, first = uniform(at.step);
    const int count = uniform(static_cast<int>(min(left, total - first)));
    left -= count;
    const bool whole = count == total, begun = first > 0;
    // the next share's place
    at.step = 0;
    if (first + count == total && ++at.tile == steps.tiles) {
      at.tile = 0;
      if (++at.kh == a.Hk) {
        at.kh = 0;
        while (++at.b < a.B && span(a, at.b).n == 0) {}
      }
    }

    const int j0 = block0 + wave * kHeld, j1 = j0 + kHeld - 1, kj = j0 + (lane & 31);
    int g = uniform(static_cast<int>(first / per));  // the head and tile that are loaded next
    int tile = uniform(block0 / R + static_cast<int>(first - static_cast<int64_t>(g) * per));
    const int tile_end = block0 / R + per;
    Staged<L> qs, ds;
    Rows qr = rows_of<T>(a.q, s.start, s.n, a.q_row, kh * group + g, a.D);
    Rows dr = rows_of<T>(a.dout, s.start, s.n, pitch, kh * group + g, a.D);
    qs.init(qr), ds.init(dr);
    float st = 0.f;
    auto load = [&]() {
      const int i0 = tile * R;
      qs.load(qr, i0), ds.load(dr, i0);
      if (threadIdx.x < 2 * R) {
        const int i = i0 + threadIdx.x % R;
        const bool lse = threadIdx.x < R;
        st = i < s.n ? (lse ? a.lse_in : parts.delta)[(s.start + i) * a.Hq + kh * group + g] * (lse ? kLog2e : 1.f) : 0.f;
      }
      if (++tile == tile_end) {
        tile = block0 / R, ++g;
        qr.base += a.D * sizeof(T), dr.base += a.D * sizeof(T);
      }
    };
    int fill = 0;
    auto store = [&](int buf) {
      qs.store(lds + fill), ds.store(lds + fill + L::BYTES);
      if (threadIdx.x < 2 * R) stat[buf][threadIdx.x / R][threadIdx.x % R] = st;
    };
    int next0 = tile * R;
    load();
    // all steps of a wave, which forms dV, dK (the second sum) or both
    auto walk = [&](auto what) {
      constexpr int WHAT = decltype(what)::value;
      constexpr bool VALUES = WHAT != kSecond, KEYS = WHAT != kFirst;
      u32x4 kf[L::KF], vf[KEYS ? L::KF : 1];
      load_held<L>(rows_of<T>(a.k, s.start, s.n, a.k_row, kh, a.D), j0, kf);
      if constexpr (KEYS) load_held<L>(rows_of<T>(a.v, s.start, s.n, a.v_row, kh, a.D), j0, vf);
      f32x16 dk[KEYS ? NT : 1], dv[VALUES ? NT : 1];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (KEYS) dk[t] = zero16();
        if constexpr (VALUES) dv[t] = zero16();
      }
      Lane<L> mine(0);
      store(0);
      for (int it = 0; it < count; ++it) {
        const int i0 = next0;
        next0 = tile * R;
        __syncthreads();
        if (it + 1 < count) load();
        fill ^= L::PAIR;
        const bool all = mask.all(i0, i0 + R - 1, j0, j1);
        const float* lse = stat[it & 1][0] + 4 * (lane >> 5);
#pragma unroll
        for (int u = 0; u < R / 32; ++u) {
          const bool none = mask.none(i0 + 32 * u, i0 + 32 * u + 31, j0, j1);
          if (ZEROS == 0 && none) continue;
          f32x16 c, dp;
          float p[16], y[16];
          if constexpr (KEYS) by_rows2<L>(mine, lds, lds + L::BYTES, 32 * u, 32 * u, kf, vf, c, dp);
          else c = by_rows<L>(mine, lds, 32 * u, kf);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(c[i], c2, -lse[32 * u + walked(i)]));
            if constexpr (KEYS) y[i] = p[i] * (dp[i] - lse[R + 32 * u + walked(i)]);
          }
          if (!all) {
            rarely();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (!mask.sees(i0 + 4 * (lane >> 5) + 32 * u + walked(i), kj)) p[i] = 0.f, y[i] = 0.f;
          }
          const int half = half_of<L, ZEROS>(none);
          if constexpr (VALUES)
            by_columns<L, NP>(dv, mine, rows_or_zeros<L, ZEROS>(mine, lds, 32 * u, L::BYTES, none), 32 * u, p, nullptr,
                              nullptr, half);
          if constexpr (KEYS)
            by_columns<L, NP>(dk, mine, rows_or_zeros<L, ZEROS>(mine, lds, 32 * u, 0, none), 32 * u, y, nullptr, nullptr,
                              half);
        }
        if (it + 1 < count) store(it + 1 & 1);
        mine.flip();
      }
      __syncthreads();  // the tiles are read
      if (!whole) {
        float* to = part_of<DP, BLOCK>(parts, blockIdx.x, !begun) + wave * kHeld * DP;
        if constexpr (KEYS) store_held<float, NT>(to, DP, dk, a.scale, DP);
        if constexpr (VALUES) store_held<float, NT>(to + BLOCK * DP, DP, dv, 1.f, DP);
      } else if (kj < s.n) {
        const int64_t to = (s.start + j0) * kp + static_cast<int64_t>(kh) * a.D;
        if constexpr (KEYS) store_held<TO, NT>(static_cast<TO*>(a.dk) + to, kp, dk, a.scale, a.D);
        if constexpr (VALUES) store_held<TO, NT>(static_cast<TO*>(a.dv) + to, kp, dv, 1.f, a.D);
      }
    };
    if constexpr (kApart<T, DP>) {
      if (wave_id() < N) walk(std::integral_constant<int, kFirst>{});
      else walk(std::integral_constant<int, kSecond>{});
    } else {
      walk(std::integral_constant<int, kBoth>{});
    }
  }
}

// A key tile that begins in share blockIdx.x and goes on in the next ones: its parts
// added in their order.  blockIdx.y: 16 keys of dK or of dV.
template <typename T, typename TO, int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Parts parts) {
  constexpr int R = El<T>::TILE, BLOCK = kHeld * kBlocks<T, DP>, UNITS = DP / 4, KEYS = 16;
  const int64_t share = share_of<R, BLOCK>(a, gridDim.x), end = share * (blockIdx.x + 1);
  const Place<R, BLOCK> at(a, end - 1);
  if (at.b >= a.B) return;
  const Span s = span(a, at.b);
  const int64_t total = static_cast<int64_t>(Steps<R, BLOCK>(s.n, a.Hq / a.Hk, a.window, a.sinks).seen(at.tile)) * (a.Hq / a.Hk);
  const int64_t begin = end - 1 - at.step;
  if (begin < end - share || begin + total <= end) return;
  // within the workspace also where offsets changed under the call
  const int more = static_cast<int>(min((begin + total - end + share - 1) / share,
                                        static_cast<int64_t>(gridDim.x - 1 - blockIdx.x)));
  const int which = blockIdx.y / (BLOCK / KEYS), key0 = blockIdx.y % (BLOCK / KEYS) * KEYS;
  const int64_t kp = static_cast<int64_t>(a.Hk) * a.D;
  for (int x = threadIdx.x; x < KEYS * UNITS; x += 256) {
    const int key = key0 + x / UNITS, d = x % UNITS * 4;
    if (at.tile * BLOCK + key >= s.n || d >= a.D) continue;
    const int64_t from = (static_cast<int64_t>(which) * BLOCK + key) * DP + d;
    float sum[4];
    ld4<float>(part_of<DP, BLOCK>(parts, blockIdx.x, true) + from, sum);
#pragma unroll 4
    for (int i = 1; i <= more; ++i) {
      float y[4];
      ld4<float>(part_of<DP, BLOCK>(parts, blockIdx.x + i, false) + from, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += y[k];
    }
    store4<TO>(static_cast<TO*>(which ? a.dv : a.dk) + (s.start + at.tile * BLOCK + key) * kp +
                   static_cast<int64_t>(at.kh) * a.D + d,
               sum);
  }
}

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

// Workgroups of the (dK, dV) kernel: as many as the card holds at once, each with
// kLeast steps or more.
constexpr int64_t kLeast = 2;
template <typename T, int DP>
int shares_for(const AttnArgs& a) {
  // a ragged batch has no more steps than its rows as sequences of the longest length
  const int64_t n = std::min(a.T, a.rows), seqs = std::min(a.B, ceil_div(a.rows, n) + 1);
  const Steps<El<T>::TILE, kHeld * kBlocks<T, DP>> s(n, a.Hq / a.Hk, a.window, a.sinks);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(256 * kResident<T, DP>, s.before(s.tiles) * a.Hk * seqs / kLeast)));
}
template <typename T, int DP>
size_t parts_of(const AttnArgs& a, int shares, Parts* p) {
  const size_t delta = (static_cast<size_t>(a.rows) * a.Hq * sizeof(float) + 255) / 256 * 256;
  p->delta = reinterpret_cast<float*>(a.ws);
  p->sums = reinterpret_cast<float*>(a.ws + delta);
  return delta + (shares > 1 ? static_cast<size_t>(shares) * 4 * kHeld * kBlocks<T, DP> * DP * sizeof(float) : 0);
}

// Whether the kernels that hold queries give each wave 32 of its own: where 128 rows of
// both tensors do not fit LDS, or from so many blocks of 128 query rows on; fewer leave
// compute units idle.  One bound for the forward and dQ of a type and width, between what
// short sequences and long ones want, whose rows differ more in length.  us, 32 of its
// own : the same 32, 8 heads, all earlier tokens visible:
//   channels    tokens  blocks  forward      dQ
//   bf16,  64      128     256    11 : 16      14 : 20
//                 2048     128    51 : 30      56 : 29
//                 2048     256    51 : 38      56 : 43
//                 2048     512    63 : 69      83 : 75
//   bf16, 128      128     256    14 : 27      20 : 42
//                 2048     128    68 : 47      91 : 55
//                 1536     192    55 : 58      75 : 70
//                 2048     256    69 : 88      97 : 105    (96 channels alike)
//   bf16, 256      128      64    19 : 18      25 : 23
//                  512      32    44 : 50      49 : 37
//                 1024      64    77 : 98      81 : 59
//                 2048     128   140 : 196    149 : 120
//   fp32,  64      128     256    20 : 34      26 : 46
//                 2048     256   166 : 137    227 : 165
//                 2048     512   288 : 268    411 : 329
//                 2048    1024   476 : 533    711 : 651
//   fp32, 128      128    1024   153 : 183    183 : 315
//                 2048     512   719 : 459    763 : 596
//                 2048    1024  1160 : 936   1304 : 1240
// At 256 channels the narrow tile has one buffer and its forward spills; so does the wide
// forward of fp32 at 128.
template <typename T, int DP> constexpr bool kNarrow = 256 * DP * sizeof(T) <= (128 << 10);
template <typename T, int DP> constexpr int64_t kWideFrom = sizeof(T) == 2 ? (DP <= 128 ? 256 : 64) : DP <= 64 ? 256 : 1024;
template <typename T, int DP>
bool wide(const AttnArgs& a) {
  return a.B * a.Hq * ceil_div(a.T, kBlock) >= kWideFrom<T, DP>;
}

template <typename T, typename TO, int DP, bool WIDE>
hipError_t fwd(const AttnArgs& a, hipStream_t st) {
  constexpr int NP = sizeof(TO) == 2 ? 2 : 3;
  ProfScope prof("attention", st);
  const dim3 grid(a.Hq, static_cast<unsigned>(ceil_div(a.T, WIDE ? kBlock : kHeld)), static_cast<unsigned>(a.B));
  attn_fwd_kernel<T, TO, DP, NP, WIDE><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}
template <typename T, typename TO, int DP>
hipError_t fwd(const AttnArgs& a, hipStream_t st) {
  if constexpr (kNarrow<T, DP>)
    if (!wide<T, DP>(a)) return fwd<T, TO, DP, false>(a, st);
  return fwd<T, TO, DP, true>(a, st);
}

template <typename T, typename TO, int DP, bool WIDE>
hipError_t dq(const AttnArgs& a, hipStream_t st) {
  constexpr int NP = sizeof(TO) == 2 ? 2 : 3;
  ProfScope prof("attention_dq", st);
  using C = Dq<T, TO, DP, WIDE>;
  const dim3 grid(a.Hq, static_cast<unsigned>(ceil_div(a.T, C::BLOCK)), static_cast<unsigned>(a.B));
  attn_dq_kernel<T, TO, DP, NP, WIDE><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}
template <typename T, typename TO, int DP>
hipError_t bwd(const AttnArgs& a, hipStream_t st) {
  constexpr int NP = sizeof(TO) == 2 ? 2 : 3;
  hipError_t e;
  if constexpr (kNarrow<T, DP>) e = wide<T, DP>(a) ? dq<T, TO, DP, true>(a, st) : dq<T, TO, DP, false>(a, st);
  else e = dq<T, TO, DP, true>(a, st);
  if (e != hipSuccess) return e;
  const int shares = shares_for<T, DP>(a);
  Parts parts;
  parts_of<T, DP>(a, shares, &parts);
  {
    ProfScope prof("attention_dkv", st);
    attn_dkv_kernel<T, TO, DP, NP><<<dim3(shares), 256, 0, st>>>(a, parts);
    if (e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (shares == 1) return hipSuccess;
  ProfScope prof("attention_join", st);
  attn_join_kernel<T, TO, DP><<<dim3(shares, 2 * kHeld * kBlocks<T, DP> / 16), 256, 0, st>>>(a, parts);
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t fwd_dim(const AttnArgs& a, hipStream_t st) {
  if (a.D <= 64) return fwd<T, TO, 64>(a, st);
  return a.D <= 128 ? fwd<T, TO, 128>(a, st) : fwd<T, TO, 256>(a, st);
}
template <typename T, typename TO>
hipError_t bwd_dim(const AttnArgs& a, hipStream_t st) {
  if (a.D <= 64) return bwd<T, TO, 64>(a, st);
  return a.D <= 128 ? bwd<T, TO, 128>(a, st) : bwd<T, TO, 256>(a, st);
}

template <typename T, int DP>
size_t workspace(const AttnArgs& a) {
  Parts p;
  return parts_of<T, DP>(a, shares_for<T, DP>(a), &p);
}
template <typename T>
size_t workspace_dim(const AttnArgs& a) {
  return a.D <= 64 ? workspace<T, 64>(a) : a.D <= 128 ? workspace<T, 128>(a) : workspace<T, 256>(a);
}

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st) {
  if (a.io_bf16) return a.out_bf16 ? fwd_dim<bf16_t, bf16_t>(a, st) : fwd_dim<bf16_t, float>(a, st);
  return a.out_bf16 ? fwd_dim<float, bf16_t>(a, st) : fwd_dim<float, float>(a, st);
}

size_t attn_bwd_workspace(const AttnArgs& a) {
  return a.io_bf16 ? workspace_dim<bf16_t>(a) : workspace_dim<float>(a);
}

hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st) {
  if (a.io_bf16) return a.out_bf16 ? bwd_dim<bf16_t, bf16_t>(a, st) : bwd_dim<bf16_t, float>(a, st);
  return a.out_bf16 ? bwd_dim<float, bf16_t>(a, st) : bwd_dim<float, float>(a, st);
}

}  // namespace gdr
