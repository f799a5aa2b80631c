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
// dQ and (dK, dV) are formed by two kernels, each in a fixed order without
// atomics.  dK and dV add up over the query heads that share a key head and over
// the queries; where there are few key tiles, or where a tile's keys are seen by
// far more queries than the others' (first tokens under a window), this axis is
// cut and the parts are joined by a third launch.
//
// Precision.  bf16 inputs are operands as they are; P and dS enter as two bf16
// operands (16 bits) for outputs in bf16 and as three for outputs in fp32: one is
// as coarse as the output itself.  fp32 inputs use fp32 products.

#include <algorithm>

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

// Element types: PER elements in 16 bytes, TILE rows walked at a time.
template <typename T> struct El;
template <> struct El<bf16_t> {
  static constexpr int PER = 8, TILE = 64;
};
template <> struct El<float> {
  static constexpr int PER = 4, TILE = 32;
};

// A tile of ROWS x DP in LDS.  Unit u (16 bytes) of a row lies at u ^ mix(row):
// rows read together by a wave's 16-lane groups fall on different banks.
template <typename T, int DP> struct Tile {
  static constexpr int PER = El<T>::PER, ROWS = El<T>::TILE, UNITS = DP / PER, KF = UNITS / 2;
  static constexpr int BYTES = ROWS * DP * sizeof(T), LOADS = ROWS * UNITS / 256;
  static __device__ __forceinline__ int mix(int row) {
    return UNITS == 8 ? ((row >> 1 & 1) << 2 | (row >> 2 & 3)) : ((row & 3) << 2 | (row >> 2 & 3));
  }
  static __device__ __forceinline__ int at(int row, int unit) { return row * UNITS * 16 + ((unit ^ mix(row)) << 4); }
};

// Rows of a tensor [.., rows, heads, D] for one sequence and head.
struct Rows {
  const char* base;     // the sequence's first row, the head's first channel
  int64_t pitch;        // bytes between rows
  int64_t n;            // rows of the sequence
};
template <typename T>
__device__ __forceinline__ Rows rows_of(const void* p, int64_t start, int64_t n, int64_t row, int head, int D) {
  return {static_cast<const char*>(p) + (start * row + static_cast<int64_t>(head) * D) * sizeof(T),
          row * static_cast<int64_t>(sizeof(T)), n};
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;
// Rows row0 .. row0 + count - 1 as a buffer: what lies past the sequence's end
// reads as zero.
__device__ __forceinline__ rsrc_t buffer(const Rows& r, int64_t row0, int count, int bytes) {
  const int64_t left = max(int64_t(0), min(r.n - row0, static_cast<int64_t>(count)));
  const int64_t first = min(row0, r.n);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(r.base) + first * r.pitch, 0,
                                           left ? static_cast<int>((left - 1) * r.pitch + bytes) : 0, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(rsrc_t b, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, static_cast<int>(at), 0, 0));
}

// A tile on its way to LDS through registers.
template <typename T, int DP> struct Staged {
  using L = Tile<T, DP>;
  u32x4 x[L::LOADS];
  __device__ __forceinline__ void load(const Rows& r, int64_t row0, int D) {
    const rsrc_t b = buffer(r, row0, L::ROWS, D * static_cast<int>(sizeof(T)));
#pragma unroll
    for (int i = 0; i < L::LOADS; ++i) {
      const int idx = threadIdx.x + 256 * i, row = idx / L::UNITS, u = idx % L::UNITS;
      x[i] = load16(b, u * L::PER < D ? static_cast<uint32_t>(row * r.pitch + u * 16) : 0x7fffffffu);
    }
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
template <typename T, int DP>
__device__ __forceinline__ void load_held(const Rows& r, int64_t row0, int D, u32x4 (&f)[Tile<T, DP>::KF]) {
  using L = Tile<T, DP>;
  const rsrc_t b = buffer(r, row0, kHeld, D * static_cast<int>(sizeof(T)));
  const int row = lane_id() & 31, h = lane_id() >> 5;
#pragma unroll
  for (int i = 0; i < L::KF; ++i)
    f[i] = load16(b, (2 * i + h) * L::PER < D ? static_cast<uint32_t>(row * r.pitch + (2 * i + h) * 16) : 0x7fffffffu);
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

// (rows row0 .. + 31 of the tile) x (held rows): lane (held row lane % 32) holds
// tile rows row0 + 8 (i / 4) + 4 (lane / 32) + i % 4.
template <typename T, int DP>
__device__ __forceinline__ f32x16 by_rows(const char* lds, int row0, const u32x4 (&held)[Tile<T, DP>::KF]) {
  using L = Tile<T, DP>;
  const int row = lane_id() & 31, h = lane_id() >> 5;
  f32x16 c = zero16();
#pragma unroll
  for (int i = 0; i < L::KF; ++i)
    c = mma<T>(*reinterpret_cast<const u32x4*>(lds + row0 * L::UNITS * 16 + L::at(row, 2 * i + h)), held[i], c);
  return c;
}
__device__ __forceinline__ int walked(int i) { return 8 * (i >> 2) + 4 * (lane_id() >> 5) + (i & 3); }

// NP bf16 parts of eight values, most significant first.
template <int NP>
__device__ __forceinline__ void split(const float* p, bf16x8 (&out)[NP]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = p[i];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const __bf16 x = static_cast<__bf16>(r);
      out[k][i] = x;
      r -= static_cast<float>(x);
    }
  }
}

// acc[t] += (channels 32 t .. + 31 of tile rows row0 .. + 31)^T x p, p as by_rows
// gives it: lane (held row) then has channels 32 t + walked(i).  With MORE, more
// += the same of y, as one bf16 operand.
template <typename T, int DP, int NP, bool MORE = false>
__device__ __forceinline__ void by_columns(f32x16 (&acc)[DP / 32], const char* lds, int row0, const float (&p)[16],
                                           f32x16* more = nullptr, const float* y = nullptr) {
  using L = Tile<T, DP>;
  const int lane = lane_id(), h = lane >> 5;
  if constexpr (sizeof(T) == 2) {
    const int q = lane & 15, side = lane >> 4 & 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bf16x8 f[NP], g[1];
      split<NP>(p + 8 * k, f);
      if constexpr (MORE) split<1>(y + 8 * k, g);
#pragma unroll
      for (int t = 0; t < DP / 32; ++t) {
        const int unit = 4 * t + 2 * side + (q >> 1 & 1), row = 4 * h + (q >> 2);
        const char* at = lds + (row0 + 16 * k) * L::UNITS * 16 + (q & 1) * 8;
        const bf16x4 a = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + L::at(row, unit))));
        const bf16x4 b = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + L::at(row + 8, unit))));
        const bf16x8 x{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
        for (int n = NP - 1; n >= 0; --n)
          acc[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, f[n], acc[t], 0, 0, 0);
        if constexpr (MORE) more[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, g[0], more[t], 0, 0, 0);
      }
    }
  } else {
    const int d = lane & 31;
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int t = 0; t < DP / 32; ++t) {
        const float x = *reinterpret_cast<const float*>(lds + row0 * L::UNITS * 16 + L::at(walked(i), 8 * t + (d >> 2)) +
                                                        (d & 3) * 4);
        acc[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, p[i], acc[t], 0, 0, 0);
        if constexpr (MORE) more[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, y[i], more[t], 0, 0, 0);
      }
  }
}

// A wave's held rows, channels 32 t + walked(i) each, times f, to rows of `out`.
template <typename TO, int DP>
__device__ __forceinline__ void store_held(TO* out, int64_t pitch, const f32x16 (&acc)[DP / 32], float f, int D) {
  TO* at = out + static_cast<int64_t>(lane_id() & 31) * pitch + 4 * (lane_id() >> 5);
#pragma unroll
  for (int t = 0; t < DP / 32; ++t)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (32 * t + 8 * b + 4 * (lane_id() >> 5) >= D) continue;
      const float x[4] = {acc[t][4 * b] * f, acc[t][4 * b + 1] * f, acc[t][4 * b + 2] * f, acc[t][4 * b + 3] * f};
      st4<TO>(at + 32 * t + 8 * b, x);
    }
}

// A sequence of the batch: its first row and its length.
struct Span {
  int64_t start, n;
};
__device__ __forceinline__ Span span(const AttnArgs& a, int64_t b) {
  if (!a.cu) return {b * a.T, a.T};
  const int64_t lo = a.cu[b];
  return {lo, max(int64_t(0), min(a.cu[b + 1] - lo, a.T))};
}

// Visible: j <= i and (no window, or i - j < window, or j < sinks).
struct Mask {
  int64_t window, sinks;
  __device__ __forceinline__ bool sees(int64_t i, int64_t j) const {
    return j <= i && (window == 0 || i - j < window || j < sinks);
  }
  // all pairs of i0 .. i1 and j0 .. j1; none of them
  __device__ __forceinline__ bool all(int64_t i0, int64_t i1, int64_t j0, int64_t j1) const {
    return j1 <= i0 && (window == 0 || i1 - j0 < window || j1 < sinks);
  }
  __device__ __forceinline__ bool none(int64_t i0, int64_t i1, int64_t j0, int64_t j1) const {
    return j0 > i1 || (window != 0 && i0 - j1 >= window && j0 >= sinks);
  }
};

// Key tiles that queries q0 .. q1 see, as a list: sinks, then the window.
struct KeyTiles {
  int64_t head, skip, count;
  __device__ __forceinline__ KeyTiles(const Mask& m, int64_t q0, int64_t q1, int tile) {
    const int64_t first = m.window == 0 ? 0 : max(int64_t(0), q0 - m.window + 1) / tile;
    head = m.window == 0 ? 0 : min((m.sinks + tile - 1) / tile, first);
    skip = first - head;
    count = q1 / tile + 1 - skip;
  }
  __device__ __forceinline__ int64_t operator[](int64_t i) const { return i < head ? i : i + skip; }
};

template <typename T, typename TO, int DP, int NP>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void attn_fwd_kernel(AttnArgs a) {
  using L = Tile<T, DP>;
  __shared__ __align__(16) char lk[2][L::BYTES];
  __shared__ __align__(16) char lv[2][L::BYTES];
  const int h = blockIdx.x, kh = h / (a.Hq / a.Hk), lane = lane_id(), wave = threadIdx.x >> 6;
  const Span s = span(a, blockIdx.z);
  const int64_t block0 = static_cast<int64_t>(gridDim.y - 1 - blockIdx.y) * kBlock;  // long rows first
  if (block0 >= s.n) return;
  const Mask mask{a.window, a.sinks};
  const int64_t block1 = min(block0 + kBlock, s.n) - 1;
  const KeyTiles tiles(mask, block0, block1, L::ROWS);
  const Rows kr = rows_of<T>(a.k, s.start, s.n, a.k_row, kh, a.D);
  const Rows vr = rows_of<T>(a.v, s.start, s.n, a.v_row, kh, a.D);
  const int64_t q0 = block0 + wave * kHeld, q1 = q0 + kHeld - 1, qi = q0 + (lane & 31);
  u32x4 qf[L::KF];
  load_held<T, DP>(rows_of<T>(a.q, s.start, s.n, a.q_row, h, a.D), q0, a.D, qf);
  f32x16 acc[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) acc[t] = zero16();
  float m = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;

  Staged<T, DP> ks, vs;
  ks.load(kr, tiles[0] * L::ROWS, a.D);
  vs.load(vr, tiles[0] * L::ROWS, a.D);
  ks.store(lk[0]);
  vs.store(lv[0]);
  for (int64_t it = 0; it < tiles.count; ++it) {
    const int buf = it & 1;
    __syncthreads();
    const bool more = it + 1 < tiles.count;
    if (more) {
      ks.load(kr, tiles[it + 1] * L::ROWS, a.D);
      vs.load(vr, tiles[it + 1] * L::ROWS, a.D);
    }
    const int64_t j0 = tiles[it] * L::ROWS;
    if (!mask.none(q0, q1, j0, j0 + L::ROWS - 1)) {
      constexpr int SUB = L::ROWS / 32;
      float x[SUB][16];
      float top = -INFINITY;
      const bool all = mask.all(q0, q1, j0, j0 + L::ROWS - 1);
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const f32x16 c = by_rows<T, DP>(lk[buf], 32 * u, qf);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[u][i] = c[i];
        if (!all)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!mask.sees(qi, j0 + 32 * u + walked(i))) x[u][i] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, x[u][i]);
      }
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      if (__any(top > m)) {
        top = fmaxf(top, m);
        const float f = m == -INFINITY ? 0.f : exp2f((m - top) * c2);
        l *= f;
#pragma unroll
        for (int t = 0; t < DP / 32; ++t) acc[t] *= f;
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
        by_columns<T, DP, NP>(acc, lv[buf], 32 * u, x[u]);
      }
    }
    if (more) {
      ks.store(lk[buf ^ 1]);
      vs.store(lv[buf ^ 1]);
    }
  }
  l += __shfl_xor(l, 32, 64);
  if (qi >= s.n) return;
  const int64_t pitch = static_cast<int64_t>(a.Hq) * a.D;
  store_held<TO, DP>(static_cast<TO*>(a.o) + (s.start + q0) * pitch + static_cast<int64_t>(h) * a.D, pitch, acc,
                     1.f / l, a.D);
  if (lane < 32) a.lse[(s.start + qi) * a.Hq + h] = fmaf(m, a.scale, log2f(l) * kLn2);
}

// dQ, and delta into the workspace (the next kernel reads it).
//
// delta = dO . O with an O rounded to bf16 is off by 2^-9 of its terms, more than
// dS itself where one key has most of a row's weight.  So with a bf16 O the sum of
// dS over the keys, which is 0 for the right delta, is what delta is off by (e):
// dQ has e (P K) taken off (K^T is in registers for dS; one bf16 operand for P is
// enough, as e is small), and the delta that is passed on has e added.
template <typename T, typename TO, int DP, int NP>
__global__ __launch_bounds__(256, 1) void attn_dq_kernel(AttnArgs a) {
  using L = Tile<T, DP>;
  __shared__ __align__(16) char lk[L::BYTES];
  __shared__ __align__(16) char lv[L::BYTES];
  const int h = blockIdx.x, kh = h / (a.Hq / a.Hk), lane = lane_id(), wave = threadIdx.x >> 6;
  const Span s = span(a, blockIdx.z);
  const int64_t block0 = static_cast<int64_t>(gridDim.y - 1 - blockIdx.y) * kBlock;
  if (block0 >= s.n) return;
  const Mask mask{a.window, a.sinks};
  const KeyTiles tiles(mask, block0, min(block0 + kBlock, s.n) - 1, L::ROWS);
  const Rows kr = rows_of<T>(a.k, s.start, s.n, a.k_row, kh, a.D);
  const Rows vr = rows_of<T>(a.v, s.start, s.n, a.v_row, kh, a.D);
  const int64_t q0 = block0 + wave * kHeld, q1 = q0 + kHeld - 1, qi = q0 + (lane & 31);
  const int64_t pitch = static_cast<int64_t>(a.Hq) * a.D;
  Staged<T, DP> ks, vs;
  ks.load(kr, tiles[0] * L::ROWS, a.D);
  vs.load(vr, tiles[0] * L::ROWS, a.D);
  u32x4 qf[L::KF], df[L::KF];
  load_held<T, DP>(rows_of<T>(a.q, s.start, s.n, a.q_row, h, a.D), q0, a.D, qf);
  load_held<T, DP>(rows_of<T>(a.dout, s.start, s.n, pitch, h, a.D), q0, a.D, df);
  float lse2 = 0.f, delta = 0.f;
  if (qi < s.n) {
    lse2 = a.lse_in[(s.start + qi) * a.Hq + h] * kLog2e;
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
  constexpr bool FIX = sizeof(TO) == 2;
  f32x16 acc[DP / 32], pk[FIX ? DP / 32 : 1];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) {
    acc[t] = zero16();
    if constexpr (FIX) pk[t] = zero16();
  }
  float off = 0.f;
  const float c2 = a.scale * kLog2e;
  for (int64_t it = 0; it < tiles.count; ++it) {
    ks.store(lk);
    vs.store(lv);
    __syncthreads();
    if (it + 1 < tiles.count) {
      ks.load(kr, tiles[it + 1] * L::ROWS, a.D);
      vs.load(vr, tiles[it + 1] * L::ROWS, a.D);
    }
#pragma unroll
    for (int u = 0; u < L::ROWS / 32; ++u) {
      const int64_t j0 = tiles[it] * L::ROWS + 32 * u;
      if (mask.none(q0, q1, j0, j0 + 31)) continue;
      const bool all = mask.all(q0, q1, j0, j0 + 31);
      const f32x16 c = by_rows<T, DP>(lk, 32 * u, qf);
      const f32x16 dp = by_rows<T, DP>(lv, 32 * u, df);
      float x[16], p[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        p[i] = __builtin_amdgcn_exp2f(fmaf(c[i], c2, -lse2));
        x[i] = p[i] * (dp[i] - delta);
        if (!all && !mask.sees(qi, j0 + walked(i))) x[i] = 0.f, p[i] = 0.f;
        off += x[i];
      }
      by_columns<T, DP, NP, FIX>(acc, lk, 32 * u, x, pk, p);
    }
    __syncthreads();
  }
  if constexpr (FIX) {
    off += __shfl_xor(off, 32, 64);
    delta += off;
#pragma unroll
    for (int t = 0; t < DP / 32; ++t) acc[t] -= off * pk[t];
  }
  if (qi >= s.n) return;
  if (lane < 32) reinterpret_cast<float*>(a.ws)[(s.start + qi) * a.Hq + h] = delta;
  store_held<TO, DP>(static_cast<TO*>(a.dq) + (s.start + q0) * pitch + static_cast<int64_t>(h) * a.D, pitch, acc,
                     a.scale, a.D);
}

// How the queries that a key tile is seen by are cut: `parts` for each tile, and
// `first` for the first `sink_tiles` tiles under a window.
struct Cut {
  int tiles, sink_tiles, parts, first;
};
// Partial sums: [part][row][Hk][D] of dK, then of dV; of the first tiles'
// [part][sequence][row][Hk][D] likewise.
struct Parts {
  float *delta, *rest, *first;
};

template <typename T, typename TO, int DP, int NP>
__global__ __launch_bounds__(256, 1) void attn_dkv_kernel(AttnArgs a, Cut cut, Parts parts) {
  using L = Tile<T, DP>;
  __shared__ __align__(16) char lq[L::BYTES];
  __shared__ __align__(16) char ld[L::BYTES];
  __shared__ __align__(16) float stat[2][L::ROWS];
  const int kh = blockIdx.y, group = a.Hq / a.Hk, lane = lane_id(), wave = threadIdx.x >> 6;
  const Span s = span(a, blockIdx.z);
  const bool early = static_cast<int>(blockIdx.x) < cut.sink_tiles * cut.first;
  const int job = early ? blockIdx.x : blockIdx.x - cut.sink_tiles * cut.first;
  const int of = early ? cut.first : cut.parts, part = job % of;
  const int64_t block0 = static_cast<int64_t>(job / of + (early ? 0 : cut.sink_tiles)) * kBlock;
  if (block0 >= s.n) return;
  const Mask mask{a.window, a.sinks};
  const int64_t j0 = block0 + wave * kHeld, j1 = j0 + kHeld - 1, kj = j0 + (lane & 31);
  // query tiles that see the keys, for each head of the group
  const int64_t last = mask.window == 0 || block0 < mask.sinks ? s.n - 1
                                                               : min(s.n - 1, block0 + kBlock - 1 + mask.window - 1);
  const int64_t tile0 = block0 / L::ROWS, per = last / L::ROWS - tile0 + 1, total = per * group;
  const int64_t it0 = total * part / of, it1 = total * (part + 1) / of;

  u32x4 kf[L::KF], vf[L::KF];
  load_held<T, DP>(rows_of<T>(a.k, s.start, s.n, a.k_row, kh, a.D), j0, a.D, kf);
  load_held<T, DP>(rows_of<T>(a.v, s.start, s.n, a.v_row, kh, a.D), j0, a.D, vf);
  f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int t = 0; t < DP / 32; ++t) dk[t] = zero16(), dv[t] = zero16();
  const float c2 = a.scale * kLog2e;
  const int64_t pitch = static_cast<int64_t>(a.Hq) * a.D;
  Staged<T, DP> qs, ds;
  float st = 0.f;
  auto load = [&](int64_t it) {
    const int g = static_cast<int>(it / per);
    const int64_t i0 = (tile0 + it - g * per) * L::ROWS;
    const int h = kh * group + g;
    qs.load(rows_of<T>(a.q, s.start, s.n, a.q_row, h, a.D), i0, a.D);
    ds.load(rows_of<T>(a.dout, s.start, s.n, pitch, h, a.D), i0, a.D);
    if (threadIdx.x < 2 * L::ROWS) {
      const int64_t i = i0 + threadIdx.x % L::ROWS;
      const bool lse = threadIdx.x < L::ROWS;
      st = i < s.n ? (lse ? a.lse_in : parts.delta)[(s.start + i) * a.Hq + h] * (lse ? kLog2e : 1.f) : 0.f;
    }
  };
  if (it0 < it1) load(it0);
  for (int64_t it = it0; it < it1; ++it) {
    qs.store(lq);
    ds.store(ld);
    if (threadIdx.x < 2 * L::ROWS) stat[threadIdx.x / L::ROWS][threadIdx.x % L::ROWS] = st;
    __syncthreads();
    if (it + 1 < it1) load(it + 1);
#pragma unroll
    for (int u = 0; u < L::ROWS / 32; ++u) {
      const int64_t i0 = (tile0 + it % per) * L::ROWS + 32 * u;
      if (mask.none(i0, i0 + 31, j0, j1)) continue;
      const bool all = mask.all(i0, i0 + 31, j0, j1);
      const f32x16 c = by_rows<T, DP>(lq, 32 * u, kf);
      const f32x16 dp = by_rows<T, DP>(ld, 32 * u, vf);
      float p[16], x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = 32 * u + walked(i);
        p[i] = __builtin_amdgcn_exp2f(fmaf(c[i], c2, -stat[0][r]));
        x[i] = p[i] * (dp[i] - stat[1][r]);
        if (!all && !mask.sees(i0 + walked(i), kj)) p[i] = 0.f, x[i] = 0.f;
      }
      by_columns<T, DP, NP>(dv, ld, 32 * u, p);
      by_columns<T, DP, NP>(dk, lq, 32 * u, x);
    }
    __syncthreads();
  }
  if (kj >= s.n) return;
  const int64_t kp = static_cast<int64_t>(a.Hk) * a.D, at = static_cast<int64_t>(kh) * a.D;
  if (of == 1) {
    store_held<TO, DP>(static_cast<TO*>(a.dk) + (s.start + j0) * kp + at, kp, dk, a.scale, a.D);
    store_held<TO, DP>(static_cast<TO*>(a.dv) + (s.start + j0) * kp + at, kp, dv, 1.f, a.D);
    return;
  }
  const int64_t rows = early ? a.B * cut.sink_tiles * kBlock : a.rows;
  const int64_t row = early ? static_cast<int64_t>(blockIdx.z) * cut.sink_tiles * kBlock + j0 : s.start + j0;
  float* to = (early ? parts.first : parts.rest) + (part * rows + row) * kp + at;
  store_held<float, DP>(to, kp, dk, a.scale, a.D);
  store_held<float, DP>(to + of * rows * kp, kp, dv, 1.f, a.D);
}

// The parts of a key tile added, in their order.
template <typename TO>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, Cut cut, Parts parts) {
  const Span s = span(a, blockIdx.z);
  const int64_t tile = blockIdx.x, block0 = tile * kBlock;
  const bool early = tile < cut.sink_tiles;
  const int of = early ? cut.first : cut.parts;
  if (block0 >= s.n || of == 1) return;
  const int64_t kp = static_cast<int64_t>(a.Hk) * a.D, at = static_cast<int64_t>(blockIdx.y) * a.D;
  const int64_t rows = early ? a.B * cut.sink_tiles * kBlock : a.rows;
  const int64_t row = early ? static_cast<int64_t>(blockIdx.z) * cut.sink_tiles * kBlock + block0 : s.start + block0;
  const float* from = (early ? parts.first : parts.rest) + row * kp + at;
  const int n = static_cast<int>(min(s.n - block0, static_cast<int64_t>(kBlock))), units = a.D / 4;
  for (int x = threadIdx.x; x < 2 * n * units; x += 256) {
    const int which = x / (n * units), r = x / units % n, d = x % units * 4;
    const float* p = from + which * of * rows * kp + r * kp + d;
    float sum[4] = {};
#pragma unroll 4
    for (int i = 0; i < of; ++i) {
      float y[4];
      ld4<float>(p + i * rows * kp, y);
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += y[k];
    }
    st4<TO>(static_cast<TO*>(which ? a.dv : a.dk) + (s.start + block0 + r) * kp + at + d, sum);
  }
}

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }

constexpr int64_t kFill = 512;  // workgroups that fill the card
constexpr int kMaxParts = 64;
Cut cut_of(const AttnArgs& a) {
  const int tile = a.io_bf16 ? El<bf16_t>::TILE : El<float>::TILE;
  Cut c{};
  c.tiles = static_cast<int>(ceil_div(a.T, kBlock));
  c.sink_tiles = a.window ? static_cast<int>(std::min<int64_t>(ceil_div(a.sinks, kBlock), c.tiles)) : 0;
  const int64_t reach = a.window ? std::min(a.T, a.window + kBlock) : a.T;
  const int64_t group = a.Hq / a.Hk, steps = ceil_div(reach, tile) * group, all = ceil_div(a.T, tile) * group;
  const int64_t blocks = std::max<int64_t>(1, a.B * a.Hk * c.tiles);
  c.parts = static_cast<int>(std::max<int64_t>(1, std::min({ceil_div(kFill, blocks), ceil_div(steps, 4),
                                                            static_cast<int64_t>(kMaxParts)})));
  // the first tiles' queries are cut as finely as the others', while there are few
  // such tiles
  const int64_t firsts = std::max<int64_t>(1, a.B * a.Hk * c.sink_tiles);
  c.first = static_cast<int>(std::max<int64_t>(
      1, std::min({ceil_div(c.parts * all, steps), ceil_div(2 * kFill, firsts), static_cast<int64_t>(kMaxParts)})));
  return c;
}
size_t parts_of(const AttnArgs& a, const Cut& c, char* ws, Parts* p) {
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t kp = static_cast<size_t>(a.Hk) * a.D * sizeof(float);
  size_t at = 0;
  p->delta = reinterpret_cast<float*>(ws);
  at += up(static_cast<size_t>(a.rows) * a.Hq * sizeof(float));
  p->rest = reinterpret_cast<float*>(ws + at);
  if (c.parts > 1 && c.tiles > c.sink_tiles) at += up(2 * kp * c.parts * a.rows);
  p->first = reinterpret_cast<float*>(ws + at);
  if (c.first > 1 && c.sink_tiles) at += up(2 * kp * c.first * a.B * c.sink_tiles * kBlock);
  return at;
}

template <typename T, typename TO, int DP>
hipError_t fwd(const AttnArgs& a, hipStream_t st) {
  constexpr int NP = sizeof(TO) == 2 ? 2 : 3;
  ProfScope prof("attention", st);
  const dim3 grid(a.Hq, static_cast<unsigned>(ceil_div(a.T, kBlock)), static_cast<unsigned>(a.B));
  attn_fwd_kernel<T, TO, DP, NP><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <typename T, typename TO, int DP>
hipError_t bwd(const AttnArgs& a, hipStream_t st) {
  constexpr int NP = sizeof(TO) == 2 ? 2 : 3;
  const Cut cut = cut_of(a);
  Parts parts;
  parts_of(a, cut, a.ws, &parts);
  {
    ProfScope prof("attention_dq", st);
    const dim3 grid(a.Hq, static_cast<unsigned>(cut.tiles), static_cast<unsigned>(a.B));
    attn_dq_kernel<T, TO, DP, NP><<<grid, 256, 0, st>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  {
    ProfScope prof("attention_dkv", st);
    const dim3 grid(cut.sink_tiles * cut.first + (cut.tiles - cut.sink_tiles) * cut.parts, a.Hk,
                    static_cast<unsigned>(a.B));
    attn_dkv_kernel<T, TO, DP, NP><<<grid, 256, 0, st>>>(a, cut, parts);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  const int joined = cut.parts > 1 ? cut.tiles : cut.first > 1 ? cut.sink_tiles : 0;
  if (!joined) return hipSuccess;
  ProfScope prof("attention_join", st);
  attn_join_kernel<TO><<<dim3(joined, a.Hk, static_cast<unsigned>(a.B)), 256, 0, st>>>(a, cut, parts);
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

}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st) {
  if (a.io_bf16) return a.out_bf16 ? fwd_dim<bf16_t, bf16_t>(a, st) : fwd_dim<bf16_t, float>(a, st);
  return a.out_bf16 ? fwd_dim<float, bf16_t>(a, st) : fwd_dim<float, float>(a, st);
}

size_t attn_bwd_workspace(const AttnArgs& a) {
  Parts p;
  return parts_of(a, cut_of(a), nullptr, &p);
}

hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st) {
  if (a.io_bf16) return a.out_bf16 ? bwd_dim<bf16_t, bf16_t>(a, st) : bwd_dim<bf16_t, float>(a, st);
  return a.out_bf16 ? bwd_dim<float, bf16_t>(a, st) : bwd_dim<float, float>(a, st);
}

}  // namespace gdr
