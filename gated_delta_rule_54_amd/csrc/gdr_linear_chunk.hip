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
// One workgroup of four waves walks a segment of a sequence for one value
// head and a slice of columns; a wave keeps its 16 NCT columns of H in
// accumulators for the whole walk.  The accumulator layout of H (rows 4g + e
// of a 16-row tile in lane group g) is at the same time the operand layout of
// X H when X's columns are read in the matching order, so H never leaves the
// registers; O is formed transposed, so that a lane stores 4 consecutive
// columns of one token.  X, Y and Z pass through LDS (X and Y are shared by
// the waves, Y and Z are read transposed); the next chunk is loaded into
// registers while this one is worked on.
//
// Precision.  bf16 inputs are matrix-core operands as they are.  What is
// computed on the way (P, H, the decayed Z) is fp32: where a result is
// returned in fp32, or a sum over all tokens is (the state; the terms of the
// decay's gradient), it enters the product as a sum of three bf16 values (24
// bits); otherwise, for an output that is rounded to bf16 itself, as one.
// fp32 inputs use fp32 operands.

#include <algorithm>
#include <type_traits>

#include "gdr_device.h"
#include "gdr_linear.h"

namespace gdr {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
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

// log2 of a token's decay factor.  A factor below 2^-185 is zero in every
// product; the bound keeps -Inf out of the differences of sums.
__device__ __forceinline__ double log2_decay(float g) {
  return (g < -128.f ? -128.0 : static_cast<double>(g)) * 1.4426950408889634;
}

// Matrix-core operands: lane group g holds steps 8g .. 8g + 7 of a 32-step
// block of the summed index.  C chunk rows, PAD elements between LDS rows.
struct OpB {
  using E = uint16_t;
  static constexpr int C = 64, PAD = 8, PER = 8;  // PER: elements of a 16-byte unit
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
  static __device__ __forceinline__ f32x4 mma(F a, F b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ void widen(float (&x)[8], F f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(f[i]);
  }
  // x as a sum of NS operands
  template <int NS>
  static __device__ __forceinline__ void split(F (&f)[NS], const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float r = x[i];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        f[s][i] = static_cast<__bf16>(r);
        if (s + 1 < NS) r -= static_cast<float>(f[s][i]);
      }
    }
  }
  // x[0..3] into NS tiles, `step` elements apart, at p
  template <int NS>
  static __device__ __forceinline__ void put4(E* p, int step, f32x4 x) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      bf16x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = static_cast<__bf16>(x[i]);
        x[i] -= static_cast<float>(v[i]);
      }
      *reinterpret_cast<bf16x4*>(p + s * step) = v;
    }
  }
};

struct OpF {
  using E = float;
  static constexpr int C = 32, PAD = 4, PER = 4;
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
  template <int NS>
  static __device__ __forceinline__ void put4(E* p, int, f32x4 x) {
    *reinterpret_cast<f32x4*>(p) = x;
  }
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, uint32_t nbytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(nbytes), 0x00020000);
}

// A chunk's rows of one tensor as a buffer that ends with them: row i of the
// chunk lies i rows from its start, or, backward in time, n - 1 - i.  Reads
// outside give zeros, writes are dropped: rows at or past n lie beyond the end
// either way (backward as negative offsets, which wrap around), and kNone does.
constexpr uint32_t kNone = 0xf0000000u;
struct Rows {
  const char* at;  // row 0 of the segment's walk
  uint32_t rowb;   // bytes between tokens; a chunk's rows span less than 2^30 bytes
  uint32_t width;  // bytes of a row that may be touched
  bool rev;
  __device__ __forceinline__ rsrc_t chunk(int64_t first, int n) const {
    const char* lo = rev ? at - (first + n - 1) * rowb : at + first * rowb;
    return make_rsrc(lo, (n - 1) * rowb + width);
  }
  // Offset of row i, from the chunk's n = C form.
  __device__ __forceinline__ uint32_t row(int i, int C) const { return (rev ? C - 1 - i : i) * rowb; }
  __device__ __forceinline__ uint32_t shift(int n, int C) const { return rev ? (C - n) * rowb : 0; }
};

// Rows of a chunk on their way from memory to LDS: 16-byte unit e of the
// [C][W] tile is loaded by thread e % 256 in round e / 256.
template <typename OP, int W>
struct Stage {
  static constexpr int UPR = W / OP::PER, N = OP::C * UPR / 256, STEP = 256 / UPR;
  static_assert(OP::C * UPR % 256 == 0, "whole rounds");
  Rows rows;
  uint32_t off;  // of round 0
  bool on;       // the thread's columns exist
  u32x4 r[N];
  __device__ __forceinline__ void init(const Rows& t) {
    rows = t;
    on = 16 * (threadIdx.x % UPR) < t.width;
    off = rows.row(threadIdx.x / UPR, OP::C) + 16 * (threadIdx.x % UPR);
  }
  __device__ __forceinline__ void load(int64_t first, int n) {
    const rsrc_t b = rows.chunk(first, n);
    const uint32_t o = off - rows.shift(n, OP::C), step = rows.rev ? -(STEP * rows.rowb) : STEP * rows.rowb;
#pragma unroll
    for (int u = 0; u < N; ++u) r[u] = __builtin_amdgcn_raw_buffer_load_b128(b, on ? o + u * step : kNone, 0, 0);
  }
  __device__ __forceinline__ void store(typename OP::E* dst) const {
    typename OP::E* p = dst + threadIdx.x / UPR * (W + OP::PAD) + OP::PER * (threadIdx.x % UPR);
#pragma unroll
    for (int u = 0; u < N; ++u) *reinterpret_cast<u32x4*>(p + u * STEP * (W + OP::PAD)) = r[u];
  }
};

constexpr int kW2 = kLinSlice;  // columns of a workgroup's slice: 16 for each of its four waves

template <typename OP, int D1P>
struct Tiles {
  static constexpr int C = OP::C, LD1 = D1P + OP::PAD, LDZ = kW2 + OP::PAD, LDP = C + OP::PAD;
};

// Decay factors of a chunk's rows.
template <int C>
struct Decay {
  double A[C];             // log2, running
  float fo[C], fz[C];      // 2^A_i, 2^(A_C - A_i)
  float all;               // 2^A_C
};

// Where a workgroup works.
struct Walk {
  LinChain c;
  int64_t b, bh, seg, row0;  // row0: the segment's first token row
  int64_t t0, len;           // the segment's first token in its sequence, its length
  int h, col0, sl;
  bool first, last;          // of the sequence's segments, in the chain's direction
};

// One walk over a segment.  NS: operands that P and H enter the output's
// products as; STATE: only the state is wanted.  `total` (in the last wave):
// the segment's log2 decay.
//
// Two barriers a chunk.  Between the first and the second the waves read X, Y,
// Z and write P; behind the second they read P and write the next chunk's
// X, Y, Z.  A wave forms the column block of P that has its index, from X
// fragments that it needs for X H anyway.
template <typename OP, int D1P, int NS, bool STATE>
__device__ __forceinline__ void walk(const LinChains& a, const Walk& w, f32x4 (&H)[D1P / 16], double& total,
                                     typename OP::E* Xs, typename OP::E* Ys, typename OP::E* Zs, typename OP::E* Ps,
                                     Decay<OP::C>* Ds, float (*Es)[OP::C]) {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  using F = typename OP::F;
  constexpr int C = T::C, NI = C / 16, KB = D1P / 32, KS = C / 32, LD1 = T::LD1, LDZ = T::LDZ, LDP = T::LDP;
  constexpr int NU = std::is_same_v<OP, OpB> ? 3 : 1;  // operands the state's update enters as
  constexpr uint32_t ES = sizeof(E);
  const LinChain& c = w.c;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g4 = 4 * (lane >> 4);
  const int wc = 16 * wave;  // the wave's first column in the slice
  const bool rev = c.rev;
  const int64_t start = w.row0 + (rev ? w.len - 1 : 0);
  const int w2 = min(c.D2 - w.col0, kW2);
  auto rows = [&](const void* p, int64_t stride, int group, int D, int col, int width) {
    const char* at = static_cast<const char*>(p) + (start * stride + static_cast<int64_t>(w.h / group) * D + col) * ES;
    return Rows{at, static_cast<uint32_t>(stride) * ES, width * ES, rev};
  };
  Stage<OP, D1P> sx, sy;
  Stage<OP, kW2> sz;
  if constexpr (!STATE) sx.init(rows(c.x, c.xr, c.xg, c.D1, 0, c.D1));
  sy.init(rows(c.y, c.yr, c.yg, c.D1, 0, c.D1));
  sz.init(rows(c.z, c.zr, c.zg, c.D2, w.col0, w2));
  // output rows, and those of e's other factor
  const bool wide = c.out_partial || !a.out_bf16, has = wc < w2;
  const uint32_t os = wide ? 4 : 2;
  Rows ro{}, re{};
  uint32_t oo = 0, oe = 0;
  if constexpr (!STATE) {
    const int64_t orow = c.out_partial ? w.b * a.T + w.t0 + (rev ? w.len - 1 : 0) : start;
    ro = Rows{static_cast<char*>(c.out) + ((orow * a.Hv + w.h) * c.D2 + w.col0) * os,
              static_cast<uint32_t>(a.Hv) * c.D2 * os, w2 * os, rev};
    oo = ro.row(m, C) + (wc + g4) * os;
    if (c.ex) {
      re = rows(c.ex, c.er, c.eg, c.D2, w.col0, w2);
      oe = re.row(m, C) + (wc + g4) * ES;
    }
  }
  const float* gp = a.g ? a.g + w.h + (a.head_decay ? 0 : start * a.Hv) : nullptr;
  const int64_t gstep = a.head_decay ? 0 : rev ? -a.Hv : a.Hv;

  float gn = 0.f;
  auto fetch = [&](int64_t at) {
    const int n = static_cast<int>(min(w.len - at, static_cast<int64_t>(C)));
    if constexpr (!STATE) sx.load(at, n);
    sy.load(at, n);
    sz.load(at, n);
    if (wave == 3) gn = gp && lane < n ? gp[(at + lane) * gstep] : 0.f;
  };
  auto put = [&]() {
    if constexpr (!STATE) sx.store(Xs);
    sy.store(Ys);
    sz.store(Zs);
  };
  auto decays = [&](Decay<C>& d) {  // by the last wave
    const double g2 = log2_decay(gn), inc = prefix64(g2), A = rev ? inc - g2 : inc, all = __shfl(inc, 63, 64);
    if (lane < C) {
      d.A[lane] = A;
      d.fo[lane] = __builtin_amdgcn_exp2f(static_cast<float>(A));
      d.fz[lane] = __builtin_amdgcn_exp2f(static_cast<float>(all - A));
    }
    if (lane == 0) d.all = __builtin_amdgcn_exp2f(static_cast<float>(all));
    total += all;
  };
  total = 0.0;
  fetch(0);
  put();
  if (wave == 3) decays(Ds[0]);
  __syncthreads();

  int buf = 0;
  for (int64_t at = 0; at < w.len; at += C, buf ^= 1) {
    const int n = static_cast<int>(min(w.len - at, static_cast<int64_t>(C)));
    const bool more = at + C < w.len;
    const Decay<C>& d = Ds[buf];
    if (more) fetch(at + C);

    f32x4 O[NI];
    if constexpr (!STATE) {
      // X H, and the wave's block of P; both transposed
      f32x4 S[NI];
#pragma unroll
      for (int ib = 0; ib < NI; ++ib) O[ib] = S[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        F hf[NS];
        const f32x4 h0 = H[2 * kb], h1 = H[2 * kb + 1];
        const float x[8] = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
        OP::template split<NS>(hf, x);
        const F yf = OP::run(Ys + (16 * (wave % NI) + m) * LD1 + 32 * kb + 2 * g4);
#pragma unroll
        for (int ib = 0; ib < NI; ++ib) {
          const F xf = OP::run(Xs + (16 * ib + m) * LD1 + 32 * kb + 2 * g4);
          if (ib >= wave) S[ib] = OP::mma(yf, xf, S[ib]);
#pragma unroll
          for (int s = NS - 1; s >= 0; --s) O[ib] = OP::mma(hf[s], xf, O[ib]);
        }
      }
      // P = S o 2^(A_i - A_j): the lane holds rows j .. j + 3 of column i
      if (wave < NI) {
        const int j = 16 * wave + g4;
        double Aj[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) Aj[e] = d.A[j + e];
#pragma unroll
        for (int ib = 0; ib < NI; ++ib)
          if (ib >= wave) {
            const int i = 16 * ib + m;
            const double Ai = d.A[i];
            f32x4 p;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = j + e <= i ? S[ib][e] * __builtin_amdgcn_exp2f(static_cast<float>(Ai - Aj[e])) : 0.f;
            OP::template put4<NS>(Ps + i * LDP + j, C * LDP, p);
          }
      }
    }

    // Z as it is for the output, decayed to the chunk's end for the state
    F zf[KS], zu[KS][NU];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      zf[ks] = OP::col(Zs, LDZ, 32 * ks, wc, 4);
      float x[8];
      OP::widen(x, zf[ks]);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= d.fz[32 * ks + 2 * g4 + i];
      OP::template split<NU>(zu[ks], x);
    }
    const float ft = d.all;
#pragma unroll
    for (int t = 0; t < D1P / 16; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) H[t][e] *= ft;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        // tile t holds rows 32 (t / 2) + 8 g + 4 (t % 2) + e, the order of X's operands
        const F yf = OP::col(Ys, LD1, 32 * ks, 32 * (t / 2) + 4 * (t % 2), 8);
#pragma unroll
        for (int s = NU - 1; s >= 0; --s) H[t] = OP::mma(yf, zu[ks][s], H[t]);
      }
    }
    if constexpr (!STATE) {
#pragma unroll
      for (int ib = 0; ib < NI; ++ib) {
        const float f = d.fo[16 * ib + m];
#pragma unroll
        for (int e = 0; e < 4; ++e) O[ib][e] *= f;
      }
    }
    if (more && wave == 3) decays(Ds[buf ^ 1]);
    __syncthreads();
    if (more) put();

    if constexpr (!STATE) {
      rsrc_t be;
      if (c.ex) be = re.chunk(at, n);
      float ex[NI][4];
      if (c.ex) {
        const uint32_t step = rev ? -(16 * re.rowb) : 16 * re.rowb, at0 = oe - re.shift(n, C);
#pragma unroll
        for (int ib = 0; ib < NI; ++ib) {
          const uint32_t o = has ? at0 + ib * step : kNone;
          if constexpr (ES == 2) {
            const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(be, o, 0, 0);
            ex[ib][0] = __uint_as_float(u[0] << 16), ex[ib][1] = __uint_as_float(u[0] & 0xffff0000u);
            ex[ib][2] = __uint_as_float(u[1] << 16), ex[ib][3] = __uint_as_float(u[1] & 0xffff0000u);
          } else {
            const u32x4 u = __builtin_amdgcn_raw_buffer_load_b128(be, o, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) ex[ib][e] = __uint_as_float(static_cast<unsigned>(u[e]));
          }
        }
      }
      // O += P Z
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int ib = 2 * ks; ib < NI; ++ib)
#pragma unroll
          for (int s = NS - 1; s >= 0; --s)
            O[ib] = OP::mma(zf[ks], OP::run(Ps + s * C * LDP + (16 * ib + m) * LDP + 32 * ks + 2 * g4), O[ib]);
      const rsrc_t bo = ro.chunk(at, n);
      const uint32_t step = rev ? -(16 * ro.rowb) : 16 * ro.rowb, at0 = oo - ro.shift(n, C);
#pragma unroll
      for (int ib = 0; ib < NI; ++ib) {
        const uint32_t o = has ? at0 + ib * step : kNone;
        if (wide) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[ib]), bo, o, 0, 0);
        } else {
          const bf16x4 v{static_cast<__bf16>(O[ib][0]), static_cast<__bf16>(O[ib][1]), static_cast<__bf16>(O[ib][2]),
                         static_cast<__bf16>(O[ib][3])};
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), bo, o, 0, 0);
        }
        if (c.ex) {
          const float e = rows4_sum((ex[ib][0] * O[ib][0] + ex[ib][1] * O[ib][1]) +
                                    (ex[ib][2] * O[ib][2] + ex[ib][3] * O[ib][3]));
          if (lane < 16) Es[wave][16 * ib + m] = e;
        }
      }
    }
    __syncthreads();
    if constexpr (!STATE) {
      if (c.ex && tid < n) {
        const int64_t t = rev ? w.t0 + w.len - 1 - at - tid : w.t0 + at + tid;
        c.e[(w.sl * a.B * a.Hv + w.bh) * a.T + t] = (Es[0][tid] + Es[1][tid]) + (Es[2][tid] + Es[3][tid]);
      }
    }
  }
}

// Logical index of this workgroup: each of the 8 XCDs takes a contiguous
// range, so that the workgroups that read the same rows share an L2.
__device__ __forceinline__ int64_t xcd_index() {
  const int64_t per = (static_cast<int64_t>(gridDim.x) + 7) / 8;
  return static_cast<int64_t>(blockIdx.x % 8) * per + blockIdx.x / 8;
}

// Finds the workgroup's place; false: nothing to do.  Slices are fastest (of
// all chains of a head), then heads, then sequences, then segments.
__device__ __forceinline__ bool find(const LinChains& a, Walk& w) {
  const int n0 = lin_slices(a.c[0].D2), n1 = a.n > 1 ? lin_slices(a.c[1].D2) : 0,
            n2 = a.n > 2 ? lin_slices(a.c[2].D2) : 0, all = n0 + n1 + n2;
  const int64_t k = xcd_index();
  int s = static_cast<int>(k % all);
  const int64_t r = k / all;
  if (r >= a.B * a.Hv * a.segments) return false;
  const int ci = s < n0 ? 0 : s < n0 + n1 ? 1 : 2;
  s -= ci == 0 ? 0 : ci == 1 ? n0 : n0 + n1;
  w.c = lin_chain(a, ci);
  w.sl = s;
  w.col0 = s * kW2;
  w.bh = r % (a.B * a.Hv);
  w.seg = r / (a.B * a.Hv);
  w.h = static_cast<int>(w.bh % a.Hv);
  w.b = w.bh / a.Hv;
  const LinSpan sp = lin_span(a.cu, w.b, a.T);
  w.t0 = w.seg * a.seg;
  if (w.t0 >= sp.len && w.seg > 0) return false;
  w.len = min(a.seg, sp.len - w.t0);
  w.row0 = sp.t0 + w.t0;
  const bool begin = w.seg == 0, end = w.t0 + w.len >= sp.len;
  w.first = w.c.rev ? end : begin;
  w.last = w.c.rev ? begin : end;
  return true;
}

// Element (d1, d2) of a state for the lane's accumulator tile t (rows d1 ..
// d1 + 3 are its elements).
template <int D1P, typename F>
__device__ __forceinline__ void each_state(const LinChain& c, int col0, F&& f) {
  const int lane = lane_id(), d2 = col0 + 16 * static_cast<int>(threadIdx.x >> 6) + (lane & 15);
#pragma unroll
  for (int t = 0; t < D1P / 16; ++t) {
    const int d1 = 32 * (t / 2) + 8 * (lane >> 4) + 4 * (t % 2);
    if (d2 < c.D2 && d1 < c.D1) f(t, static_cast<int64_t>(d1) * c.s1 + static_cast<int64_t>(d2) * c.s2);
  }
}

template <typename OP, int D1P, int NS0, int NS1>
__global__ __launch_bounds__(256, D1P <= 128 ? 2 : 1) void lin_chunk_kernel(LinChains a) {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  constexpr int C = T::C, NSM = NS0 > NS1 ? NS0 : NS1;
  __shared__ __align__(16) E Xs[C * T::LD1], Ys[C * T::LD1], Zs[C * T::LDZ], Ps[NSM * C * T::LDP];
  __shared__ __align__(16) Decay<C> Ds[2];
  __shared__ __align__(16) float Es[4][C];
  Walk w;
  if (!find(a, w)) return;
  const LinChain& c = w.c;
  const int64_t one = static_cast<int64_t>(c.D1) * c.D2;
  // the blocks of P above the diagonal that a 32-step product reads stay zero
  for (int e = threadIdx.x; e < NSM * C * T::LDP; e += 256) Ps[e] = E(0);

  f32x4 H[D1P / 16];
#pragma unroll
  for (int t = 0; t < D1P / 16; ++t) H[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* in = c.seg_in ? c.seg_in + (w.bh * a.segments + w.seg) * one : c.s_in ? c.s_in + w.bh * one : nullptr;
  if (in)
    each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
      for (int e = 0; e < 4; ++e) H[t][e] = in[at + static_cast<int64_t>(e) * c.s1];
    });
  double total;
  if (w.len > 0) {
    if (NS0 == NS1 || c.exact) walk<OP, D1P, NS0, false>(a, w, H, total, Xs, Ys, Zs, Ps, Ds, Es);
    else walk<OP, D1P, NS1, false>(a, w, H, total, Xs, Ys, Zs, Ps, Ds, Es);
  }
  if (c.xdot) {
    const float* dot = c.seg_dot ? c.seg_dot + (w.bh * a.segments + w.seg) * one : c.dot ? c.dot + w.bh * one : nullptr;
    float s = 0.f;
    if (dot)
      each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s += H[t][e] * dot[at + static_cast<int64_t>(e) * c.s1];
      });
    s = rows4_sum(row16_sum(s));
    __syncthreads();
    if (lane_id() == 0) Es[threadIdx.x >> 6][0] = s;
    __syncthreads();
    if (threadIdx.x == 0)
      c.xdot[(w.seg * a.B * a.Hv + w.bh) * lin_slices(c.D2) + w.sl] =
          (Es[0][0] + Es[1][0]) + (Es[2][0] + Es[3][0]);
  }
  if (c.s_out && w.last) {
    float* out = c.s_out + w.bh * one;
    each_state<D1P>(c, w.col0, [&](int t, int64_t at) {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[at + static_cast<int64_t>(e) * c.s1] = H[t][e];
    });
  }
}

// Every segment's own contribution to the state at its end (in the chain's
// direction), from zero.  The last segment's is not needed.  The chain forward
// in time leaves the segments' factors, but the last one's, which only the
// chain backward in time needs and leaves.
template <typename OP, int D1P>
__global__ __launch_bounds__(256, 2) void lin_segment_kernel(LinChains a, float* factor) {
  using T = Tiles<OP, D1P>;
  using E = typename OP::E;
  constexpr int C = T::C;
  __shared__ __align__(16) E Ys[C * T::LD1], Zs[C * T::LDZ];
  __shared__ __align__(16) Decay<C> Ds[2];
  Walk w;
  if (!find(a, w) || w.last) return;
  const LinChain& c = w.c;
  const int64_t one = static_cast<int64_t>(c.D1) * c.D2;
  f32x4 H[D1P / 16];
#pragma unroll
  for (int t = 0; t < D1P / 16; ++t) H[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  double total;
  walk<OP, D1P, 1, true>(a, w, H, total, nullptr, Ys, Zs, nullptr, Ds, nullptr);
  const int64_t at0 = w.bh * a.segments + w.seg;
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

// Cutting sequences: workgroups wanted in the launch, the shortest segment.
#ifndef TG
#define TG 512
#endif
#ifndef MS
#define MS 256
#endif
constexpr int64_t kTargetGroups = TG, kMinSegment = MS;

int64_t chunk_blocks(const LinChains& a) {
  int64_t all = 0;
  for (int i = 0; i < a.n; ++i) all += lin_slices(a.c[i].D2);
  return (all * a.B * a.Hv * a.segments + 7) / 8 * 8;
}

int max_d1(const LinChains& a) {
  int d = 0;
  for (int i = 0; i < a.n; ++i) d = std::max(d, a.c[i].D1);
  return d;
}

template <typename OP, int D1P>
hipError_t run_chunks(const LinChains& a, bool exact, bool mixed, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(chunk_blocks(a)));
  if constexpr (std::is_same_v<OP, OpF>) {
    lin_chunk_kernel<OP, D1P, 1, 1><<<grid, 256, 0, st>>>(a);
  } else {
    if (mixed) lin_chunk_kernel<OP, D1P, 3, 1><<<grid, 256, 0, st>>>(a);
    else if (exact) lin_chunk_kernel<OP, D1P, 3, 3><<<grid, 256, 0, st>>>(a);
    else lin_chunk_kernel<OP, D1P, 1, 1><<<grid, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <typename OP, int D1P>
hipError_t run_segments(const LinChains& a, float* factor, hipStream_t st) {
  lin_segment_kernel<OP, D1P><<<static_cast<unsigned>(chunk_blocks(a)), 256, 0, st>>>(a, factor);
  return hipGetLastError();
}

// Calls f with the operand type and the padded width (an integral constant).
template <typename F>
hipError_t by_type(bool io_bf16, int d1, F&& f) {
  auto width = [&](auto op) {
    if (d1 <= 64) return f(op, std::integral_constant<int, 64>{});
    if (d1 <= 128) return f(op, std::integral_constant<int, 128>{});
    return f(op, std::integral_constant<int, 256>{});
  };
  return io_bf16 ? width(OpB{}) : width(OpF{});
}

}  // namespace

// One direction's segment states, then their factors.
LinPlan lin_plan(const LinShape& s, bool backward) {
  LinPlan p{};
  const int slices = backward ? 2 * lin_slices(s.Dk) + lin_slices(s.Dv) : lin_slices(s.Dv);
  const int64_t heads = std::max<int64_t>(1, s.B * s.Hv);
  const int64_t groups = heads * slices;
  const int64_t want = (kTargetGroups + groups - 1) / groups, most = (s.T + kMinSegment - 1) / kMinSegment;
  const int64_t n = std::max<int64_t>(1, std::min(want, most));
  p.seg = std::max<int64_t>(64, ((s.T + n - 1) / n + 63) / 64 * 64);
  p.segments = std::max<int64_t>(1, (s.T + p.seg - 1) / p.seg);
  if (p.segments > 1) {
    const size_t bh = static_cast<size_t>(s.B) * s.Hv * p.segments;
    p.states = bh * s.Dk * s.Dv * sizeof(float);
    p.bytes = (backward ? 2 : 1) * p.states + (bh * sizeof(float) + 255) / 256 * 256;
  }
  return p;
}

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
  a.c[0].exact = !s.out_bf16;
  return by_type(s.io_bf16, s.Dk, [&](auto op, auto d1) {
    return run_chunks<decltype(op), decltype(d1)::value>(a, !s.out_bf16, false, st);
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
  const bool all = !s.out_bf16, some = args.dg != nullptr;
  a.c[0].exact = a.c[1].exact = all || some;
  a.c[2].exact = all;
  {
    ProfScope prof("linear_chunks_vjp", st);
    const hipError_t e = by_type(s.io_bf16, max_d1(a), [&](auto op, auto d1) {
      return run_chunks<decltype(op), decltype(d1)::value>(a, all, some && !all, st);
    });
    if (e != hipSuccess) return e;
  }
  return launch_lin_bwd_tail(s, args, parts, p.segments, p.seg, st);
}

}  // namespace gdr
