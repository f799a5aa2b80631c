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

// Matrix-core operands: 8 consecutive steps of the summed index per lane, as
// 4 + 4 of a 32-step block; C chunk rows, PAD elements between LDS rows.
struct OpB {
  using E = uint16_t;
  static constexpr int C = 64, PAD = 8, PER = 8;  // PER: elements of a 16-byte unit
  typedef bf16x8 F;
  // row r, columns c .. c+3 and c+16 .. c+19
  static __device__ __forceinline__ F pair(const E* p) {
    const bf16x4 a = *reinterpret_cast<const bf16x4*>(p), b = *reinterpret_cast<const bf16x4*>(p + 16);
    return F{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  static __device__ __forceinline__ F run(const E* p) { return *reinterpret_cast<const F*>(p); }
  // Rows k0 + 8g .. +7 of column n0 + lane % 16 of a row-major tile: one
  // transposing read hands a group of 16 lanes 4 rows of 16 columns.
  static __device__ __forceinline__ F col(const E* M, int ld, int k0, int n0) {
    const int p = lane_id() & 15, g = lane_id() >> 4;
    const E* at = M + (k0 + 8 * g + (p >> 2)) * ld + n0 + 4 * (p & 3);
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
  static __device__ __forceinline__ F pair(const E* p) {
    F f;
#pragma unroll
    for (int i = 0; i < 4; ++i) f.v[i] = p[i], f.v[4 + i] = p[16 + i];
    return f;
  }
  static __device__ __forceinline__ F run(const E* p) {
    F f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = p[i];
    return f;
  }
  static __device__ __forceinline__ F col(const E* M, int ld, int k0, int n0) {
    const E* at = M + (k0 + 8 * (lane_id() >> 4)) * ld + n0 + (lane_id() & 15);
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

// Rows of a chunk on their way from memory to LDS: 16-byte unit e of the
// [C][W] tile is loaded by thread e % 256 in round e / 256.  Rows at or past n
// and columns at or past `units` read as zeros (their loads go to the first
// row and column instead).
template <typename OP, int W>
struct Stage {
  static constexpr int UPR = W / OP::PER, N = (OP::C * UPR + 255) / 256;
  uint4 r[N];
  __device__ __forceinline__ void load(const char* base, int64_t row_bytes, int n, int units) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int e = 256 * u + threadIdx.x, row = e / UPR, cu = e % UPR;
      const bool ok = row < n && cu < units;
      const uint4 x = *reinterpret_cast<const uint4*>(base + (ok ? row * row_bytes + 16 * cu : 0));
      r[u] = ok ? x : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void store(typename OP::E* dst) const {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int e = 256 * u + threadIdx.x, row = e / UPR, cu = e % UPR;
      if (OP::C * UPR % 256 == 0 || row < OP::C)
        *reinterpret_cast<uint4*>(dst + row * (W + OP::PAD) + OP::PER * cu) = r[u];
    }
  }
};

// The tile (i, j) of index t in the order (0,0) (1,0) (1,1) (2,0) ...
__device__ __forceinline__ int tri_row(int t) { return t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3; }

template <typename OP, int D1P, int NCT>
struct Tiles {
  static constexpr int C = OP::C, LD1 = D1P + OP::PAD, W2 = 64 * NCT, LDZ = W2 + OP::PAD, LDP = C + OP::PAD;
  static constexpr int MAXNS = std::is_same_v<OP, OpB> ? 3 : 1;
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
// products as; STATE: only the state is wanted.
template <typename OP, int D1P, int NCT, int NS, bool STATE>
__device__ __forceinline__ void walk(const LinChains& a, const Walk& w, f32x4 (&H)[NCT][D1P / 16], double& total,
                                     typename OP::E* Xs, typename OP::E* Ys, typename OP::E* Zs, typename OP::E* Ps,
                                     double* As, float* fo, float* fz, float* ftot, float (*Es)[OP::C]) {
  using T = Tiles<OP, D1P, NCT>;
  using E = typename OP::E;
  using F = typename OP::F;
  constexpr int C = T::C, NI = C / 16, KB = D1P / 32, KS = C / 32, LD1 = T::LD1, LDZ = T::LDZ, LDP = T::LDP;
  constexpr int NU = std::is_same_v<OP, OpB> ? 3 : 1;  // operands the state's update enters as
  constexpr int ES = static_cast<int>(sizeof(E));
  const LinChain& c = w.c;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int m = lane & 15, g4 = 4 * (lane >> 4);
  const int wc = 16 * NCT * wave;  // the wave's first column in the slice
  const int64_t dir = c.rev ? -1 : 1;
  const int64_t start = w.row0 + (c.rev ? w.len - 1 : 0);
  const char* xb = static_cast<const char*>(c.x) + (start * c.xr + static_cast<int64_t>(w.h / c.xg) * c.D1) * ES;
  const char* yb = static_cast<const char*>(c.y) + (start * c.yr + static_cast<int64_t>(w.h / c.yg) * c.D1) * ES;
  const char* zb =
      static_cast<const char*>(c.z) + (start * c.zr + static_cast<int64_t>(w.h / c.zg) * c.D2 + w.col0) * ES;
  const int64_t xrb = dir * c.xr * ES, yrb = dir * c.yr * ES, zrb = dir * c.zr * ES;
  const int u1 = c.D1 / OP::PER, u2 = min(c.D2 - w.col0, T::W2) / OP::PER;
  const float* gp = a.g ? a.g + w.h + (a.head_decay ? 0 : start * a.Hv) : nullptr;
  const int64_t gstep = a.head_decay ? 0 : dir * a.Hv;

  Stage<OP, D1P> sx, sy;
  Stage<OP, T::W2> sz;
  float gn = 0.f;
  auto fetch = [&](int64_t at) {
    const int n = static_cast<int>(min(w.len - at, static_cast<int64_t>(C)));
    if constexpr (!STATE) sx.load(xb + at * xrb, xrb, n, u1);
    sy.load(yb + at * yrb, yrb, n, u1);
    sz.load(zb + at * zrb, zrb, n, u2);
    if (wave == 0) gn = gp && lane < n ? gp[(at + lane) * gstep] : 0.f;
  };
  fetch(0);
  total = 0.0;

  for (int64_t at = 0; at < w.len; at += C) {
    const int n = static_cast<int>(min(w.len - at, static_cast<int64_t>(C)));
    if constexpr (!STATE) sx.store(Xs);
    sy.store(Ys);
    sz.store(Zs);
    if (wave == 0) {
      const double g2 = log2_decay(gn), inc = prefix64(g2), A = c.rev ? inc - g2 : inc;
      const double all = __shfl(inc, 63, 64);
      if (lane < C) {
        As[lane] = A;
        fo[lane] = __builtin_amdgcn_exp2f(static_cast<float>(A));
        fz[lane] = __builtin_amdgcn_exp2f(static_cast<float>(all - A));
      }
      if (lane == 0) ftot[0] = __builtin_amdgcn_exp2f(static_cast<float>(all));
      total += all;
    }
    __syncthreads();
    if (at + C < w.len) fetch(at + C);

    f32x4 O[NCT][NI];
    if constexpr (!STATE) {
      // P, transposed tiles: lane holds rows j = 16 jb + g4 + e of column i = 16 ib + m
      for (int t = wave; t < NI * (NI + 1) / 2; t += 4) {
        const int ib = tri_row(t), jb = t - ib * (ib + 1) / 2;
        f32x4 s{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
          s = OP::mma(OP::pair(Ys + (16 * jb + m) * LD1 + 32 * kb + g4),
                      OP::pair(Xs + (16 * ib + m) * LD1 + 32 * kb + g4), s);
        const int i = 16 * ib + m, j = 16 * jb + g4;
        const double Ai = As[i];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[e] = j + e <= i ? s[e] * __builtin_amdgcn_exp2f(static_cast<float>(Ai - As[j + e])) : 0.f;
        OP::template put4<NS>(Ps + i * LDP + j, C * LDP, s);
      }
      // e^{A_i} X H, transposed
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
        for (int ib = 0; ib < NI; ++ib) O[ct][ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        F hf[NCT][NS];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
          const f32x4 h0 = H[ct][2 * kb], h1 = H[ct][2 * kb + 1];
          const float x[8] = {h0[0], h0[1], h0[2], h0[3], h1[0], h1[1], h1[2], h1[3]};
          OP::template split<NS>(hf[ct], x);
        }
#pragma unroll
        for (int ib = 0; ib < NI; ++ib) {
          const F xf = OP::pair(Xs + (16 * ib + m) * LD1 + 32 * kb + g4);
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int s = NS - 1; s >= 0; --s) O[ct][ib] = OP::mma(hf[ct][s], xf, O[ct][ib]);
        }
      }
#pragma unroll
      for (int ib = 0; ib < NI; ++ib) {
        const float f = fo[16 * ib + m];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[ct][ib][e] *= f;
      }
      __syncthreads();
    }

    // Z as it is for the output, decayed to the chunk's end for the state
    F zu[KS][NCT][NU];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fz[32 * ks + 2 * g4 + i];
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) {
        const F z = OP::col(Zs, LDZ, 32 * ks, wc + 16 * ct);
        if constexpr (!STATE) {
#pragma unroll
          for (int ib = 2 * ks; ib < NI; ++ib)
#pragma unroll
            for (int s = NS - 1; s >= 0; --s)
              O[ct][ib] = OP::mma(z, OP::run(Ps + s * C * LDP + (16 * ib + m) * LDP + 32 * ks + 2 * g4), O[ct][ib]);
        }
        float x[8];
        OP::widen(x, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= f[i];
        OP::template split<NU>(zu[ks][ct], x);
      }
    }
    const float ft = ftot[0];
#pragma unroll
    for (int t = 0; t < D1P / 16; ++t) {
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e) H[ct][t][e] *= ft;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const F yf = OP::col(Ys, LD1, 32 * ks, 16 * t);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int s = NU - 1; s >= 0; --s) H[ct][t] = OP::mma(yf, zu[ks][ct][s], H[ct][t]);
      }
    }

    if constexpr (!STATE) {
#pragma unroll
      for (int ib = 0; ib < NI; ++ib) {
        const int i = 16 * ib + m;
        const int64_t row = start + dir * (at + i);
        float e = 0.f;
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
          const int col = w.col0 + wc + 16 * ct + g4;
          if (i < n && col < c.D2) {
            const float v[4] = {O[ct][ib][0], O[ct][ib][1], O[ct][ib][2], O[ct][ib][3]};
            const int64_t orow = c.out_partial ? w.b * a.T + (row - w.row0 + w.t0) : row;
            const int64_t o = (orow * a.Hv + w.h) * c.D2 + col;
            if (c.out_partial || !a.out_bf16) {
              *reinterpret_cast<f32x4*>(static_cast<float*>(c.out) + o) = O[ct][ib];
            } else {
              const bf16x4 q{static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1]), static_cast<__bf16>(v[2]),
                             static_cast<__bf16>(v[3])};
              *reinterpret_cast<bf16x4*>(static_cast<__bf16*>(c.out) + o) = q;
            }
            if (c.ex) {
              float x[4];
              ld4<E>(static_cast<const E*>(c.ex) + row * c.er + static_cast<int64_t>(w.h / c.eg) * c.D2 + col, x);
              e += (x[0] * v[0] + x[1] * v[1]) + (x[2] * v[2] + x[3] * v[3]);
            }
          }
        }
        if (c.ex) {
          e = rows4_sum(e);
          if (lane < 16) Es[wave][i] = e;
        }
      }
    }
    __syncthreads();
    if constexpr (!STATE) {
      if (c.ex && tid < n) {
        const int64_t t = c.rev ? w.t0 + w.len - 1 - at - tid : w.t0 + at + tid;
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
template <int W2>
__device__ __forceinline__ bool find(const LinChains& a, Walk& w) {
  const int n0 = lin_slices(a.c[0].D2, W2), n1 = a.n > 1 ? lin_slices(a.c[1].D2, W2) : 0,
            n2 = a.n > 2 ? lin_slices(a.c[2].D2, W2) : 0, all = n0 + n1 + n2;
  const int64_t k = xcd_index();
  int s = static_cast<int>(k % all);
  const int64_t r = k / all;
  if (r >= a.B * a.Hv * a.segments) return false;
  const int ci = s < n0 ? 0 : s < n0 + n1 ? 1 : 2;
  s -= ci == 0 ? 0 : ci == 1 ? n0 : n0 + n1;
  w.c = lin_chain(a, ci);
  w.sl = s;
  w.col0 = s * W2;
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

// Element (d1, d2) of a state for lane's accumulator element e of tile t.
template <int D1P, int NCT, typename F>
__device__ __forceinline__ void each_state(const LinChain& c, int col0, F&& f) {
  const int lane = lane_id(), wave = threadIdx.x >> 6, m = lane & 15, g4 = 4 * (lane >> 4);
#pragma unroll
  for (int ct = 0; ct < NCT; ++ct) {
    const int d2 = col0 + 16 * (NCT * wave + ct) + m;
#pragma unroll
    for (int t = 0; t < D1P / 16; ++t) {
      const int d1 = 16 * t + g4;
      if (d2 < c.D2 && d1 < c.D1) f(ct, t, static_cast<int64_t>(d1) * c.s1 + static_cast<int64_t>(d2) * c.s2);
    }
  }
}

template <typename OP, int D1P, int NCT, int NS0, int NS1>
__global__ __launch_bounds__(256) void lin_chunk_kernel(LinChains a) {
  using T = Tiles<OP, D1P, NCT>;
  using E = typename OP::E;
  constexpr int C = T::C, NSM = NS0 > NS1 ? NS0 : NS1;
  __shared__ __align__(16) E Xs[C * T::LD1], Ys[C * T::LD1], Zs[C * T::LDZ], Ps[NSM * C * T::LDP];
  __shared__ __align__(16) double As[C];
  __shared__ __align__(16) float fo[C], fz[C], ftot[1], Es[4][C];
  Walk w;
  if (!find<T::W2>(a, w)) return;
  const LinChain& c = w.c;
  const int64_t one = static_cast<int64_t>(c.D1) * c.D2;
  // the blocks of P above the diagonal that a 32-step product reads
  for (int e = threadIdx.x; e < NSM * C * T::LDP; e += 256) Ps[e] = E(0);

  f32x4 H[NCT][D1P / 16];
#pragma unroll
  for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
    for (int t = 0; t < D1P / 16; ++t) H[ct][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float* in = c.seg_in ? c.seg_in + (w.bh * a.segments + w.seg) * one : c.s_in ? c.s_in + w.bh * one : nullptr;
  if (in)
    each_state<D1P, NCT>(c, w.col0, [&](int ct, int t, int64_t at) {
#pragma unroll
      for (int e = 0; e < 4; ++e) H[ct][t][e] = in[at + static_cast<int64_t>(e) * c.s1];
    });
  double total;
  if (w.len > 0) {
    if (NS0 == NS1 || c.exact)
      walk<OP, D1P, NCT, NS0, false>(a, w, H, total, Xs, Ys, Zs, Ps, As, fo, fz, ftot, Es);
    else
      walk<OP, D1P, NCT, NS1, false>(a, w, H, total, Xs, Ys, Zs, Ps, As, fo, fz, ftot, Es);
  }
  if (c.xdot) {
    const float* dot = c.seg_dot ? c.seg_dot + (w.bh * a.segments + w.seg) * one : c.dot ? c.dot + w.bh * one : nullptr;
    float s = 0.f;
    if (dot)
      each_state<D1P, NCT>(c, w.col0, [&](int ct, int t, int64_t at) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s += H[ct][t][e] * dot[at + static_cast<int64_t>(e) * c.s1];
      });
    s = rows4_sum(row16_sum(s));
    __syncthreads();
    if (lane_id() == 0) Es[threadIdx.x >> 6][0] = s;
    __syncthreads();
    if (threadIdx.x == 0)
      c.xdot[(w.seg * a.B * a.Hv + w.bh) * lin_slices(c.D2, T::W2) + w.sl] =
          (Es[0][0] + Es[1][0]) + (Es[2][0] + Es[3][0]);
  }
  if (c.s_out && w.last) {
    float* out = c.s_out + w.bh * one;
    each_state<D1P, NCT>(c, w.col0, [&](int ct, int t, int64_t at) {
#pragma unroll
      for (int e = 0; e < 4; ++e) out[at + static_cast<int64_t>(e) * c.s1] = H[ct][t][e];
    });
  }
}

// Every segment's own contribution to the state at its end (in the chain's
// direction), from zero.  The last segment's is not needed.  The chain forward
// in time leaves the segments' factors, but the last one's, which only the
// chain backward in time needs and leaves.
template <typename OP, int D1P, int NCT>
__global__ __launch_bounds__(256) void lin_segment_kernel(LinChains a, float* factor) {
  using T = Tiles<OP, D1P, NCT>;
  using E = typename OP::E;
  constexpr int C = T::C;
  __shared__ __align__(16) E Ys[C * T::LD1], Zs[C * T::LDZ];
  __shared__ __align__(16) double As[C];
  __shared__ __align__(16) float fo[C], fz[C], ftot[1];
  Walk w;
  if (!find<T::W2>(a, w) || w.last) return;
  const LinChain& c = w.c;
  const int64_t one = static_cast<int64_t>(c.D1) * c.D2;
  f32x4 H[NCT][D1P / 16];
#pragma unroll
  for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
    for (int t = 0; t < D1P / 16; ++t) H[ct][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  double total = 0.0;
  if (w.len > 0) walk<OP, D1P, NCT, 1, true>(a, w, H, total, nullptr, Ys, Zs, nullptr, As, fo, fz, ftot, nullptr);
  const int64_t at0 = w.bh * a.segments + w.seg;
  if ((!c.rev || w.first) && w.sl == 0 && threadIdx.x == 0)
    factor[at0] = __builtin_amdgcn_exp2f(static_cast<float>(total));
  float* out = c.s_out + at0 * one;
  each_state<D1P, NCT>(c, w.col0, [&](int ct, int t, int64_t at) {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[at + static_cast<int64_t>(e) * c.s1] = H[ct][t][e];
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

// Cutting sequences: workgroups wanted in the launch, the shortest segment,
// and whether slices of 128 columns are taken where that saves workgroups.
constexpr int64_t kTargetGroups = 512, kMinSegment = 256;
constexpr int kWide = 1;

int64_t chunk_blocks(const LinChains& a, int W2) {
  int64_t all = 0;
  for (int i = 0; i < a.n; ++i) all += lin_slices(a.c[i].D2, W2);
  return (all * a.B * a.Hv * a.segments + 7) / 8 * 8;
}

int max_d1(const LinChains& a) {
  int d = 0;
  for (int i = 0; i < a.n; ++i) d = std::max(d, a.c[i].D1);
  return d;
}

template <typename OP, int D1P, int NCT>
hipError_t run_chunks(const LinChains& a, bool exact, bool mixed, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(chunk_blocks(a, 64 * NCT)));
  if constexpr (std::is_same_v<OP, OpF>) {
    lin_chunk_kernel<OP, D1P, NCT, 1, 1><<<grid, 256, 0, st>>>(a);
  } else {
    if (mixed) lin_chunk_kernel<OP, D1P, NCT, 3, 1><<<grid, 256, 0, st>>>(a);
    else if (exact) lin_chunk_kernel<OP, D1P, NCT, 3, 3><<<grid, 256, 0, st>>>(a);
    else lin_chunk_kernel<OP, D1P, NCT, 1, 1><<<grid, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

template <typename OP, int D1P, int NCT>
hipError_t run_segments(const LinChains& a, float* factor, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(chunk_blocks(a, 64 * NCT)));
  lin_segment_kernel<OP, D1P, NCT><<<grid, 256, 0, st>>>(a, factor);
  return hipGetLastError();
}

// Calls f with the kernel types for a launch's operands: integral constants
// for the padded width and the column tiles per wave.
template <typename F>
hipError_t by_type(bool io_bf16, int d1, int wide, F&& f) {
  auto width = [&](auto op) {
    using OP = decltype(op);
    if (d1 <= 64) return wide ? f(op, std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{})
                              : f(op, std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (d1 <= 128) return wide ? f(op, std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{})
                               : f(op, std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
    return f(OP{}, std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  };
  return io_bf16 ? width(OpB{}) : width(OpF{});
}

}  // namespace

// One direction's segment states, then their factors.
LinPlan lin_plan(const LinShape& s, bool backward) {
  LinPlan p{};
  const int wide_slices = backward ? 2 * lin_slices(s.Dk, 128) + lin_slices(s.Dv, 128) : lin_slices(s.Dv, 128);
  const int slices = backward ? 2 * lin_slices(s.Dk) + lin_slices(s.Dv) : lin_slices(s.Dv);
  const int64_t heads = std::max<int64_t>(1, s.B * s.Hv);
  const bool can = std::max(s.Dk, s.Dv) <= 128 && wide_slices < slices;
  p.wide = can ? kWide : 0;
  const int64_t groups = heads * (p.wide ? wide_slices : slices);
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
    hipError_t e = by_type(s.io_bf16, max_d1(a), p.wide, [&](auto op, auto d1, auto nct) {
      return run_segments<decltype(op), decltype(d1)::value, decltype(nct)::value>(a, g.factor, st);
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
  return by_type(s.io_bf16, s.Dk, p.wide, [&](auto op, auto d1, auto nct) {
    return run_chunks<decltype(op), decltype(d1)::value, decltype(nct)::value>(a, !s.out_bf16, false, st);
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
    const hipError_t e = by_type(s.io_bf16, max_d1(a), p.wide, [&](auto op, auto d1, auto nct) {
      return run_chunks<decltype(op), decltype(d1)::value, decltype(nct)::value>(a, all, some && !all, st);
    });
    if (e != hipSuccess) return e;
  }
  return launch_lin_bwd_tail(s, args, parts, lin_slices(s.Dk, p.wide ? 128 : 64), p.segments, p.seg, st);
}

}  // namespace gdr
