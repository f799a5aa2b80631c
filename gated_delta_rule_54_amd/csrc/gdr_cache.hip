// Attention of one new token for each sequence over a paged cache, split over
// the cache's length and joined.
//
//     o = sum_j e^{s_j - m} v_j / l,   s_j = scale q . k_j,   l = sum_j e^{s_j - m}
//
// in one pass: every wave keeps a running maximum m, the sum l and the weighted
// sum O of its own keys, rescaled when m grows, and (m, l, O) of disjoint sets of
// keys join as O = sum_i e^{m_i - m} O_i.
//
// Layout.  A wave takes tiles of keys (32 in bf16, 16 in fp32) for up to 16
// query heads that share a key head, and needs no LDS for them.  Scores come out
// transposed (keys x queries): a lane holds 4 keys of a 16-key product for one
// query, and these are, element by element, the summed index of the product
// with V, whose order is free.  K rows are that product's operand as they lie in
// memory (16 bytes a lane); V's operand runs over keys, so a lane loads 16 bytes
// of each of its rows and transposes 8 x 8 values in its registers.
//
// Which keys are visible is a list of places without holes (sinks, then the
// window), cut evenly between the workgroups of a sequence; a page that is not
// there leaves holes, masked key by key.
//
// Precision: K and Q enter as they are; P as three bf16 operands (24 bits) for
// either output type, for the matrix cores are idle here anyway.
//
// Bound: memory, each visible row of K and V read once.

#include <algorithm>

#include "gdr_attn.h"
#include "gdr_device.h"

namespace gdr {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;
constexpr int kMaxSplits = 256;
constexpr uint32_t kNone = 0xffffffffu;  // a place without a row

// Maximum and sum over the four rows of 16 lanes.
__device__ __forceinline__ float rows4_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}

// The visible places of a sequence of n tokens: i < head is place i, i >= head
// place i + skip.
struct Visible {
  int64_t count, head, skip;
};
__device__ __forceinline__ Visible visible(const CacheAttnArgs& a, int64_t b) {
  const int64_t n = max(int64_t(0), min(a.cache.lengths[b], a.max_len));
  if (a.window == 0 || n <= a.window || a.sinks >= n - a.window) return {n, n, 0};
  return {a.sinks + a.window, a.sinks, n - a.window - a.sinks};
}

// Keys of a split: whole tiles.
__device__ __forceinline__ int64_t split_keys(int64_t count, int splits, int tile) {
  const int64_t per = (count + splits - 1) / splits;
  return (per + tile - 1) / tile * tile;
}

// The row of place index i, in 16-byte units from the buffer's start.
__device__ __forceinline__ uint32_t row_of(const CacheView& c, const Visible& vis, const int32_t* table, int64_t i,
                                           int64_t end, int per16) {
  if (i >= end) return kNone;
  const uint64_t place = static_cast<uint64_t>(i < vis.head ? i : i + vis.skip);
  const uint32_t ps = static_cast<uint32_t>(c.page_size);
  // places fit 31 + 31 bits; most fit 32, where the division is short
  const uint64_t nth = place >> 32 ? place / ps : static_cast<uint32_t>(place) / ps;
  const int64_t page = table[nth];
  if (page < 0 || page >= c.pages) return kNone;
  return static_cast<uint32_t>((page * c.page_stride + static_cast<int64_t>(place - nth * ps) * c.token_stride) /
                               per16);
}

// D rounded up to DP; a lane's run of VL channels of a V row, NC such runs.
template <typename T, int DP> struct Shape16;
template <int DP> struct Shape16<bf16_t, DP> {
  static constexpr int PER16 = 8, TILE = 32, KF = DP / 32, VL = DP >= 128 ? 8 : 4, NC = DP / (16 * VL);
};
template <int DP> struct Shape16<float, DP> {
  static constexpr int PER16 = 4, TILE = 16, KF = DP / 16, VL = 4, NC = DP / 64;
};

// Three bf16 parts of eight values, most significant first.
__device__ __forceinline__ void split3(const float (&p)[8], bf16x8 (&out)[3]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __bf16 a = static_cast<__bf16>(p[i]);
    const float r = p[i] - static_cast<float>(a);
    const __bf16 b = static_cast<__bf16>(r);
    out[0][i] = a;
    out[1][i] = b;
    out[2][i] = static_cast<__bf16>(r - static_cast<float>(b));
  }
}

template <typename T, typename TO, int DP>
__global__ __launch_bounds__(64 * kWaves) void cache_attn_kernel(CacheAttnArgs a, int splits, int qtiles) {
  using S = Shape16<T, DP>;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int VR = BF ? 8 : 4;            // V rows of a lane
  constexpr int MT = S::NC * S::VL;         // 16-channel tiles of O
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, kh = blockIdx.y / qtiles, qt = blockIdx.y % qtiles;
  const int64_t b = blockIdx.z;
  const CacheView& c = a.cache;
  const int group = a.Hq / c.Hk, D = c.D;
  const int q0 = kh * group + qt * 16, nq = min(16, group - qt * 16);
  const Visible vis = visible(a, b);
  const int64_t per = split_keys(vis.count, splits, S::TILE);
  const int64_t begin = split * per, end = min(vis.count, begin + per);
  if (begin >= end && !(split == 0 && splits == 1)) return;  // the join knows which splits are empty

  // Q as the product's second operand: lane (query col, channels of group g)
  u32x4 qf[S::KF];
  {
    const T* q = static_cast<const T*>(a.q) + b * a.q_row + static_cast<int64_t>(q0 + col) * D;
#pragma unroll
    for (int i = 0; i < S::KF; ++i) {
      const int d = (i * 4 + g) * S::PER16;
      qf[i] = col < nq && d < D ? *reinterpret_cast<const u32x4*>(q + d) : u32x4{0, 0, 0, 0};
    }
  }
  const int32_t* table = c.table + b * c.table_row;
  const char* kbase = static_cast<const char*>(a.kc) + static_cast<int64_t>(kh) * c.head_stride * sizeof(T);
  const char* vbase = static_cast<const char*>(a.vc) + static_cast<int64_t>(kh) * c.head_stride * sizeof(T);

  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  const float c2 = a.scale * kLog2e;

  constexpr int KT = S::TILE / 16;  // 16-key products of a tile
  u32x4 kf[KT][S::KF];
  u32x4 vf[VR][S::NC];
  auto load_k = [&](uint32_t rows) {
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const uint32_t r = __shfl(rows, 16 * t + col, 64);
      const char* p = kbase + static_cast<uint64_t>(r == kNone ? 0 : r) * 16;
#pragma unroll
      for (int i = 0; i < S::KF; ++i) {
        const int d = (i * 4 + g) * S::PER16;
        kf[t][i] = d < D && r != kNone ? *reinterpret_cast<const u32x4*>(p + d * sizeof(T)) : u32x4{0, 0, 0, 0};
      }
    }
  };
  // row e of lane group g: the keys that the scores' elements hold
  auto load_v = [&](uint32_t rows) {
#pragma unroll
    for (int e = 0; e < VR; ++e) {
      const uint32_t r = __shfl(rows, BF ? (e >> 2) * 16 + 4 * g + (e & 3) : 4 * g + e, 64);
      const char* p = vbase + static_cast<uint64_t>(r == kNone ? 0 : r) * 16;
#pragma unroll
      for (int i = 0; i < S::NC; ++i) {
        const int d = 16 * S::VL * i + col * S::VL;
        if constexpr (S::VL * sizeof(T) == 16) {
          vf[e][i] = d < D && r != kNone ? *reinterpret_cast<const u32x4*>(p + d * sizeof(T)) : u32x4{0, 0, 0, 0};
        } else {
          u32x2 w{0, 0};
          if (d < D && r != kNone) w = *reinterpret_cast<const u32x2*>(p + d * sizeof(T));
          vf[e][i][0] = w[0], vf[e][i][1] = w[1];
        }
      }
    }
  };

  const int64_t step = kWaves * S::TILE;
  int64_t at = begin + wave * S::TILE;
  uint32_t rows = row_of(c, vis, table, at + lane, min(end, at + S::TILE), S::PER16);
  if (at < end) load_k(rows), load_v(rows);
  while (at < end) {
    const int64_t next = at + step;
    const uint32_t rows2 = row_of(c, vis, table, next + lane, min(end, next + S::TILE), S::PER16);
    // scores: keys 16 t + 4 g + r of query col
    float s[4 * KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      f32x4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < S::KF; ++i) {
        if constexpr (BF) {
          x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf[t][i]),
                                                      __builtin_bit_cast(bf16x8, qf[i]), x, 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kf[t][i][e]), __uint_as_float(qf[i][e]), x, 0, 0,
                                                     0);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) s[4 * t + r] = x[r];
    }
    const uint64_t live = __ballot(rows != kNone);
    if (next < end) load_k(rows2);
    if (live != (S::TILE == 32 ? 0xffffffffull : 0xffffull)) {
#pragma unroll
      for (int e = 0; e < 4 * KT; ++e)
        if (!(live >> ((e >> 2) * 16 + 4 * g + (e & 3)) & 1)) s[e] = -INFINITY;
    }
    float top = s[0];
#pragma unroll
    for (int e = 1; e < 4 * KT; ++e) top = fmaxf(top, s[e]);
    top = fmaxf(m, rows4_max(top));
    if (__any(top > m)) {
      const float f = m == -INFINITY ? 0.f : exp2f((m - top) * c2);
      l *= f;
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] *= f;
      m = top;
    }
    const float mc = m == -INFINITY ? 0.f : m * c2;
    float p[4 * KT];
#pragma unroll
    for (int e = 0; e < 4 * KT; ++e) {
      p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c2, -mc));
      l += p[e];
    }
    if constexpr (BF) {
      bf16x8 pf[3];
      split3(p, pf);
#pragma unroll
      for (int i = 0; i < S::NC; ++i)
#pragma unroll
        for (int j = 0; j < S::VL; ++j) {
          u32x4 w;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = __builtin_amdgcn_perm(vf[2 * e + 1][i][j / 2], vf[2 * e][i][j / 2],
                                         j & 1 ? 0x07060302u : 0x05040100u);
          f32x4 x = acc[i * S::VL + j];
#pragma unroll
          for (int k = 2; k >= 0; --k)
            x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), pf[k], x, 0, 0, 0);
          acc[i * S::VL + j] = x;
        }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < S::NC; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[4 * i + j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(vf[e][i][j]), p[e], acc[4 * i + j],
                                                                  0, 0, 0);
    }
    if (next < end) load_v(rows2);
    rows = rows2;
    at = next;
  }

  // Join of the waves: lane (col, g) holds O of query col at channels
  // 16 VL i + (4 g + r) VL + j.
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  __shared__ float sm[kWaves][16], sl[kWaves][16];
  __shared__ float so[kWaves / 2][16][DP + 4];
  if (lane < 16) sm[wave][col] = m, sl[wave][col] = l;
  __syncthreads();
  float mt = sm[0][col];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) mt = fmaxf(mt, sm[w][col]);
  float lt = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) lt += sl[w][col] * (sm[w][col] == -INFINITY ? 0.f : exp2f((sm[w][col] - mt) * c2));
  const float f = m == -INFINITY ? 0.f : exp2f((m - mt) * c2);
#pragma unroll
  for (int half = kWaves / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int i = 0; i < S::NC; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < S::VL; ++j)
            so[wave - half][col][16 * S::VL * i + (4 * g + r) * S::VL + j] =
                acc[i * S::VL + j][r] * (half == kWaves / 2 ? f : 1.f);
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int i = 0; i < S::NC; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int j = 0; j < S::VL; ++j) {
            const float x = acc[i * S::VL + j][r];
            acc[i * S::VL + j][r] = (half == kWaves / 2 ? x * f : x) +
                                    so[wave][col][16 * S::VL * i + (4 * g + r) * S::VL + j];
          }
    }
    __syncthreads();
  }
  if (wave != 0 || col >= nq) return;
  const int64_t head = b * a.Hq + q0 + col;
  float* part = a.part + (head * splits + split) * (D + 2);
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
#pragma unroll
  for (int i = 0; i < S::NC; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int d = 16 * S::VL * i + (4 * g + r) * S::VL;
      if (d >= D) continue;
#pragma unroll
      for (int j = 0; j < S::VL; ++j) {
        const float x = acc[i * S::VL + j][r];
        if (splits == 1) st1<TO>(static_cast<TO*>(a.o) + head * D + d + j, lt == 0.f ? 0.f : x * inv);
        else part[2 + d + j] = x;
      }
    }
  if (g != 0) return;
  if (splits > 1) part[0] = mt, part[1] = lt;
  else if (a.lse) a.lse[head] = lt == 0.f ? -INFINITY : fmaf(mt, a.scale, log2f(lt) * kLn2);
}

// One query head's parts joined; a thread takes every 128th channel.
template <typename TO>
__global__ __launch_bounds__(128) void cache_join_kernel(CacheAttnArgs a, int splits, int tile) {
  __shared__ float w[kMaxSplits];
  __shared__ float total;
  const int64_t head = blockIdx.x, b = head / a.Hq;
  const int D = a.cache.D;
  const Visible vis = visible(a, b);
  const int64_t per = split_keys(vis.count, splits, tile);
  const int n = per ? static_cast<int>((vis.count + per - 1) / per) : 0;
  const float* part = a.part + head * splits * (D + 2);
  const float c2 = a.scale * kLog2e;
  if (threadIdx.x < 64) {
    float m = -INFINITY;
    for (int i = threadIdx.x; i < n; i += 64) m = fmaxf(m, part[static_cast<int64_t>(i) * (D + 2)]);
#pragma unroll
    for (int s = 1; s < 64; s *= 2) m = fmaxf(m, __shfl_xor(m, s, 64));
    float l = 0.f;
    for (int i = threadIdx.x; i < n; i += 64) {
      const float mi = part[static_cast<int64_t>(i) * (D + 2)];
      w[i] = mi == -INFINITY ? 0.f : exp2f((mi - m) * c2);
      l += w[i] * part[static_cast<int64_t>(i) * (D + 2) + 1];
    }
    l = xsum<1, 64>(l);
    if (threadIdx.x == 0) {
      total = l;
      if (a.lse) a.lse[head] = l == 0.f ? -INFINITY : fmaf(m, a.scale, log2f(l) * kLn2);
    }
  }
  __syncthreads();
  const float l = total;
  for (int d = threadIdx.x; d < D; d += 128) {
    float x = 0.f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) x += w[i] * part[static_cast<int64_t>(i) * (D + 2) + 2 + d];
    st1<TO>(static_cast<TO*>(a.o) + head * D + d, l == 0.f ? 0.f : x / l);
  }
}
// Workgroups of a sequence and key head: enough for `kFill` on the card, each
// with at least kLeast keys.
constexpr int64_t kFill = 1024, kLeast = 256;
int splits_of(const CacheAttnArgs& a) {
  const int64_t most = a.window ? std::min(a.max_len, a.window + a.sinks) : a.max_len;
  const int group = a.Hq / a.cache.Hk;
  const int64_t base = a.B * a.cache.Hk * ((group + 15) / 16);
  const int64_t n = std::min((kFill + base - 1) / std::max<int64_t>(base, 1), (most + kLeast - 1) / kLeast);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, kMaxSplits)));
}

template <typename T, typename TO, int DP>
hipError_t launch(const CacheAttnArgs& a, hipStream_t st) {
  const int splits = splits_of(a), qtiles = (a.Hq / a.cache.Hk + 15) / 16;
  const dim3 grid(splits, a.cache.Hk * qtiles, static_cast<unsigned>(a.B));
  {
    ProfScope prof("cache_attention", st);
    cache_attn_kernel<T, TO, DP><<<grid, 64 * kWaves, 0, st>>>(a, splits, qtiles);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (splits == 1) return hipSuccess;
  ProfScope prof("cache_join", st);
  cache_join_kernel<TO><<<dim3(static_cast<unsigned>(a.B * a.Hq)), 128, 0, st>>>(a, splits, Shape16<T, DP>::TILE);
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t launch_dim(const CacheAttnArgs& a, hipStream_t st) {
  if (a.cache.D <= 64) return launch<T, TO, 64>(a, st);
  return a.cache.D <= 128 ? launch<T, TO, 128>(a, st) : launch<T, TO, 256>(a, st);
}

}  // namespace

size_t cache_attn_workspace(const CacheAttnArgs& a) {
  const int splits = splits_of(a);
  if (splits == 1) return 0;
  const size_t bytes = static_cast<size_t>(a.B) * a.Hq * splits * (a.cache.D + 2) * sizeof(float);
  return (bytes + 255) / 256 * 256;
}

hipError_t launch_cache_attn(const CacheAttnArgs& a, hipStream_t st) {
  if (a.bf16) return a.out_bf16 ? launch_dim<bf16_t, bf16_t>(a, st) : launch_dim<bf16_t, float>(a, st);
  return a.out_bf16 ? launch_dim<float, bf16_t>(a, st) : launch_dim<float, float>(a, st);
}

}  // namespace gdr
