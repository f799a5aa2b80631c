// Attention of one new token for each sequence over a paged cache, split over
// the cache's length and joined.
//
//     o = sum_j e^{s_j - m} v_j / l,   s_j = scale q . k_j,   l = sum_j e^{s_j - m}
//
// in one pass: every wave keeps a running maximum m, the sum l and the weighted
// sum O of its own keys, rescaled when m grows, and (m, l, O) of disjoint sets of
// keys join as O = sum_i e^{m_i - m} O_i.
//
// Layout.  A wave takes tiles of keys (32 in bf16 up to 128 channels, else 16) for up to 16
// query heads that share a key head, and needs no LDS for them.  Scores come out
// transposed (keys x queries): a lane holds 4 keys of a 16-key product for one
// query, and these are, element by element, the summed index of the product
// with V, whose order is free.  K rows are that product's operand as they lie in
// memory (16 bytes a lane); V's operand runs over keys, so a lane loads 16 bytes
// of each of its rows and transposes up to 8 x 8 values in its registers.
//
// Which keys are visible is a list of places without holes (sinks, then the
// window); a page that is not there leaves holes, masked key by key.  The lists of
// all sequences are cut into pieces of one length, a workgroup each, so that the
// card is filled evenly whatever the lengths, which only the device knows: every
// wave adds them up and finds its piece.
//
// Precision: K and Q enter as they are; P as three bf16 operands (24 bits) for
// either output type, for the matrix cores are idle here anyway.
//
// Bound: memory, each visible row of K and V read once, past the caches.  bf16, us
// (graph of calls, rotating buffers): 131072 tokens of 8 key heads of 128, one
// sequence, 91 (5.9 TB/s; a copy of 512 MiB reaches 6.2); 64 sequences of 512 .. 8192
// tokens, 2 of 256, 109 (5.3 TB/s).  Of the latter, cut by sequence into 8 equal
// parts each: 131; in pieces of one length, a few more than the card holds at once:
// 134; cached loads: 4-10 more; the page's number loaded where it is used, so that
// every load before it is waited for: 3-5 more; 32 keys a tile at 256 channels (one
// wave on a SIMD): 146.

#include <algorithm>

#include "gdr_attn.h"
#include "gdr_cache_pieces.h"
#include "gdr_device.h"

namespace gdr {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
template <int N> using bf16xn = __bf16 __attribute__((ext_vector_type(N)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kWaves = 4;
constexpr int kMaxCut = 512;              // sequences of a batch that is cut

// Workgroups that a compute unit holds at once (the registers that a wave needs).
constexpr int held_workgroups(bool bf16, int D) { return D <= 64 ? 3 : D <= 128 || bf16 ? 2 : 1; }
constexpr uint32_t kNone = 0xffffffffu;  // a place without a row

// Maximum and sum over the four rows of 16 lanes.
__device__ __forceinline__ float rows4_max(float x) {
  x = fmaxf(x, __shfl_xor(x, 16, 64));
  return fmaxf(x, __shfl_xor(x, 32, 64));
}

// The visible places of a sequence of n tokens: i < head is place i, i >= head
// place i + skip.
struct Visible {
  int count, head, skip;
};
__device__ __forceinline__ Visible visible(const CacheAttnArgs& a, int64_t b) {
  const int n = static_cast<int>(max(int64_t(0), min(a.cache.lengths[b], a.max_len)));
  const int window = static_cast<int>(a.window), sinks = static_cast<int>(a.sinks);
  if (window == 0 || n <= window || sinks >= n - window) return {n, n, 0};
  return {sinks + window, sinks, n - window - sinks};
}

// The pieces of a batch, for each key head: `per` keys each (whole tiles), a
// sequence's last one fewer.  Rounding up gives more of them than the sum of the
// lengths does, and a few workgroups more than the card holds at once would wait
// for a whole piece: `per` grows until there are no more than `slots`, if there
// can be (`fit`).
struct Pieces {
  int per, first;  // keys; the first piece of the sequence
  int64_t b;       // the sequence that piece f belongs to; B: there are fewer
};
__device__ __forceinline__ int wave_sum(int x) {
  return __builtin_amdgcn_readlane(wave_prefix_sum(x), 63);
}
__device__ __forceinline__ Pieces find_piece(const CacheAttnArgs& a, int f, int slots, bool fit, int tile) {
  constexpr int N = kMaxCut / 64;
  const int lane = threadIdx.x & 63, B = static_cast<int>(a.B);
  uint32_t count[N], most = 0;
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    count[k] = 64 * k + lane < B ? visible(a, 64 * k + lane).count : 0;
    sum += static_cast<double>(count[k]);
    most = max(most, count[k]);
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) {
    sum += __shfl_xor(sum, s, 64);
    most = max(most, __shfl_xor(most, s, 64));
  }
  uint32_t per = piece_keys(sum, most, slots, tile);
  for (int again = 0; fit && again < 16; ++again) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (64 * k < B) n += (count[k] + per - 1) / per;
    n = wave_sum(n);
    if (n <= slots) break;
    const uint32_t up = static_cast<uint32_t>(static_cast<float>(per) * static_cast<float>(n) / static_cast<float>(slots));
    per = (max(up, per + 1) + tile - 1) / tile * tile;
  }
  int before = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (64 * k >= B) break;
    const int n = (count[k] + per - 1) / per;
    const int upto = before + wave_prefix_sum(n);
    const uint64_t past = __ballot(upto > f);
    if (past) {
      const int at = __builtin_ctzll(past);
      return {static_cast<int>(per), __shfl(upto - n, at, 64), 64 * k + at};
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return {static_cast<int>(per), 0, a.B};
}

// A place of the list in two steps, as the page's number is loaded a tile ahead of
// its use: its page (kNone as -1: past the end, or not in the cache), then the row
// in 16-byte units from the buffer's start.
struct Place {
  int32_t page;
  uint32_t slot;
};
__device__ __forceinline__ Place place_of(const CacheView& c, const Visible& vis, const int32_t* table, int i,
                                          int end) {
  if (i >= end) return {-1, 0};
  const uint32_t place = i < vis.head ? i : i + vis.skip;
  const uint32_t ps = static_cast<uint32_t>(c.page_size), nth = place / ps;
  return {table[nth], place - nth * ps};
}
__device__ __forceinline__ uint32_t row_of(const CacheView& c, const Place& p, int per16) {
  if (p.page < 0 || p.page >= c.pages) return kNone;
  return static_cast<uint32_t>((p.page * c.page_stride + p.slot * c.token_stride) / per16);
}

// Partial results of a piece and query head: O, behind them all (m, l), and behind
// those each sequence's first piece and their number.
struct Parts {
  float* sums;
  float2* stats;
  int2* pieces;
  __device__ __forceinline__ Parts(const CacheAttnArgs& a, int pieces, int64_t piece, int head) {
    const int64_t all = static_cast<int64_t>(pieces) * a.Hq;
    float2* st = reinterpret_cast<float2*>(a.part + all * a.cache.D);
    sums = a.part + (piece * a.Hq + head) * a.cache.D;
    stats = st + piece * a.Hq + head;
    this->pieces = reinterpret_cast<int2*>(st + all);
  }
};

// D rounded up to DP; a lane's run of VL channels of a V row, NC such runs.
template <typename T, int DP> struct Shape16;
template <int DP> struct Shape16<bf16_t, DP> {
  static constexpr int PER16 = 8, TILE = DP > 128 ? 16 : 32, KF = DP / 32, VL = DP >= 128 ? 8 : 4, NC = DP / (16 * VL);
};
template <int DP> struct Shape16<float, DP> {
  static constexpr int PER16 = 4, TILE = 16, KF = DP / 16, VL = 4, NC = DP / 64;
};

// Three bf16 parts of N values, most significant first.
template <int N>
__device__ __forceinline__ void split3(const float (&p)[N], bf16xn<N> (&out)[3]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const __bf16 a = static_cast<__bf16>(p[i]);
    const float r = p[i] - static_cast<float>(a);
    const __bf16 b = static_cast<__bf16>(r);
    out[0][i] = a;
    out[1][i] = b;
    out[2][i] = static_cast<__bf16>(r - static_cast<float>(b));
  }
}

template <typename T, typename TO, int DP>
__global__ __launch_bounds__(64 * kWaves, held_workgroups(sizeof(T) == 2, DP)) void cache_attn_kernel(CacheAttnArgs a, int pieces, int slots, bool fit, int qtiles) {
  using S = Shape16<T, DP>;
  constexpr bool BF = sizeof(T) == 2;
  constexpr int VR = S::TILE / 4;           // V rows of a lane
  constexpr int MT = S::NC * S::VL;         // 16-channel tiles of O
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  const int kh = blockIdx.y / qtiles, qt = blockIdx.y % qtiles;
  const CacheView& c = a.cache;
  const int group = a.Hq / c.Hk, D = c.D;
  const int q0 = kh * group + qt * 16, nq = min(16, group - qt * 16);
  // a piece, or a whole sequence where slots is 0
  int64_t b = blockIdx.x;
  int begin = 0, per = 0;
  if (slots) {
    const Pieces piece = find_piece(a, blockIdx.x, slots, fit, S::TILE);
    b = piece.b, per = piece.per, begin = (static_cast<int>(blockIdx.x) - piece.first) * per;
    if (b == a.B) return;
  }
  const Visible vis = visible(a, b);
  const int end = slots ? min(vis.count, begin + per) : vis.count;
  if (slots && begin == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    Parts(a, pieces, 0, 0).pieces[b] = make_int2(blockIdx.x, (vis.count + per - 1) / per);

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
        kf[t][i] = d < D && r != kNone ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + d * sizeof(T))) : u32x4{0, 0, 0, 0};
      }
    }
  };
  // row e of lane group g: the keys that the scores' elements hold
  auto load_v = [&](uint32_t rows) {
#pragma unroll
    for (int e = 0; e < VR; ++e) {
      const uint32_t r = __shfl(rows, (e >> 2) * 16 + 4 * g + (e & 3), 64);
      const char* p = vbase + static_cast<uint64_t>(r == kNone ? 0 : r) * 16;
#pragma unroll
      for (int i = 0; i < S::NC; ++i) {
        const int d = 16 * S::VL * i + col * S::VL;
        if constexpr (S::VL * sizeof(T) == 16) {
          vf[e][i] = d < D && r != kNone ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + d * sizeof(T))) : u32x4{0, 0, 0, 0};
        } else {
          u32x2 w{0, 0};
          if (d < D && r != kNone) w = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + d * sizeof(T)));
          vf[e][i][0] = w[0], vf[e][i][1] = w[1];
        }
      }
    }
  };

  constexpr int step = kWaves * S::TILE;
  int at = begin + wave * S::TILE;
  auto places = [&](int from) { return place_of(c, vis, table, from + lane, min(end, from + S::TILE)); };
  uint32_t rows = row_of(c, places(at), S::PER16);
  if (at < end) load_k(rows);
  Place ahead = places(at + step);
  if (at < end) load_v(rows);
  while (at < end) {
    const int next = at + step;
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
    const uint32_t rows2 = row_of(c, ahead, S::PER16);
    if (next < end) load_k(rows2);
    ahead = places(next + step);
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
      bf16xn<4 * KT> pf[3];
      split3(p, pf);
#pragma unroll
      for (int i = 0; i < S::NC; ++i)
#pragma unroll
        for (int j = 0; j < S::VL; ++j) {
          uint32_t w[2 * KT];
#pragma unroll
          for (int e = 0; e < 2 * KT; ++e)
            w[e] = __builtin_amdgcn_perm(vf[2 * e + 1][i][j / 2], vf[2 * e][i][j / 2],
                                         j & 1 ? 0x07060302u : 0x05040100u);
          f32x4 x = acc[i * S::VL + j];
#pragma unroll
          for (int k = 2; k >= 0; --k) {
            if constexpr (KT == 2)
              x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]}),
                                                          pf[k], x, 0, 0, 0);
            else
              x = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s16x4, u32x2{w[0], w[1]}),
                                                            __builtin_bit_cast(s16x4, pf[k]), x, 0, 0, 0);
          }
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
  const Parts part(a, pieces, blockIdx.x, q0 + col);
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
        if (!slots) st1<TO>(static_cast<TO*>(a.o) + head * D + d + j, lt == 0.f ? 0.f : x * inv);
      }
      if (slots)
#pragma unroll
        for (int j = 0; j < S::VL; j += 4)
          *reinterpret_cast<f32x4*>(part.sums + d + j) =
              f32x4{acc[i * S::VL + j][r], acc[i * S::VL + j + 1][r], acc[i * S::VL + j + 2][r], acc[i * S::VL + j + 3][r]};
    }
  if (g != 0) return;
  if (slots) *part.stats = make_float2(mt, lt);
  else if (a.lse) a.lse[head] = lt == 0.f ? -INFINITY : fmaf(mt, a.scale, log2f(lt) * kLn2);
}

// One query head's parts joined: every wave weighs all pieces, a thread adds 4
// channels over every (256 / (D / 4))th piece, and the threads' sums are added in
// a fixed order.
template <typename TO>
__global__ __launch_bounds__(256) void cache_join_kernel(CacheAttnArgs a, int pieces) {
  __shared__ float w[kMaxPieces];
  __shared__ __align__(16) float sum[256][4];
  const int64_t head = blockIdx.x, b = head / a.Hq;
  const int D = a.cache.D, units = D / 4, rows = 256 / units, lane = threadIdx.x & 63;
  // a sequence without a visible token has no pieces
  const int2 mine = visible(a, b).count ? Parts(a, pieces, 0, 0).pieces[b] : make_int2(0, 0);
  // within the workspace also where lengths changed under the call
  const int n = max(0, min(mine.y, min(kMaxPieces, pieces)));
  const Parts part(a, pieces, max(0, min(mine.x, pieces - n)), static_cast<int>(head - b * a.Hq));
  const float c2 = a.scale * kLog2e;
  float2 st[kMaxPieces / 64];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMaxPieces / 64; ++k) {
    st[k] = 64 * k + lane < n ? part.stats[(64 * k + lane) * a.Hq] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, st[k].x);
  }
#pragma unroll
  for (int s = 1; s < 64; s *= 2) m = fmaxf(m, __shfl_xor(m, s, 64));
  float l = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxPieces / 64; ++k) {
    const float f = st[k].x == -INFINITY ? 0.f : exp2f((st[k].x - m) * c2);
    l += f * st[k].y;
    if (threadIdx.x < 64) w[64 * k + lane] = f;
  }
  l = xsum<1, 64>(l);
  __syncthreads();
  const int u = threadIdx.x % units, r = threadIdx.x / units;
  f32x4 x{0.f, 0.f, 0.f, 0.f};
  if (r < rows) {
#pragma unroll 8
    for (int i = r; i < n; i += rows)
      x += w[i] * *reinterpret_cast<const f32x4*>(part.sums + static_cast<int64_t>(i) * a.Hq * D + 4 * u);
  }
  *reinterpret_cast<f32x4*>(sum[threadIdx.x]) = x;
  __syncthreads();
  if (r == 0) {
    for (int k = 1; k < rows; ++k) x += *reinterpret_cast<const f32x4*>(sum[k * units + u]);
    const float y[4] = {x[0] / l, x[1] / l, x[2] / l, x[3] / l}, none[4] = {};
    if (l == 0.f) st4<TO>(static_cast<TO*>(a.o) + head * D + 4 * u, none);
    else st4<TO>(static_cast<TO*>(a.o) + head * D + 4 * u, y);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[head] = l == 0.f ? -INFINITY : fmaf(m, a.scale, log2f(l) * kLn2);
}

// How a batch is cut: a workgroup for each sequence and key head where that fills
// the card many times over, where no sequence is longer than the least piece, or
// where there are so many that adding up their lengths would take longer; else as
// many pieces as the card holds at once where there are few sequences, or twice as
// many.  us, as many : twice : four times: 64 sequences of 4096 tokens, 2 heads of 256
// 96 : 108 : 121; 20 of up to 8192, 4 heads of 64, 33 : 31 : 37; 9 of up to 8192, 8
// heads of 128, 41 : 48 : 58.  Where `fit` cannot hold, twice : four times: 100 of up
// to 4096, 4 heads of 128, 106 : 109; 300 of up to 600, 8 heads of 128, 118 : 126.
struct Cut {
  int slots, qtiles;   // pieces wanted for each key head
  bool fit;
  int64_t pieces;      // there are no more than these
};
Cut cut_of(const CacheAttnArgs& a) {
  const int64_t most = a.window ? std::min(a.max_len, a.window + a.sinks) : a.max_len;
  Cut c{};
  c.qtiles = (a.Hq / a.cache.Hk + 15) / 16;
  const int64_t heads = static_cast<int64_t>(a.cache.Hk) * c.qtiles;
  const int64_t held = 256 * held_workgroups(a.bf16, a.cache.D);
  if (most <= kLeast || a.B > kMaxCut || a.B * heads >= 16 * held) return c;
  c.fit = 2 * a.B * heads <= held;
  c.slots = static_cast<int>(std::max<int64_t>(1, (c.fit ? held : 2 * held) / heads));
  // rounding up gives each sequence a piece more; the rounds of `fit` only take away
  c.pieces = std::min(c.slots + 2 * a.B, a.B * ((most + kLeast - 1) / kLeast));
  return c;
}

template <typename T, typename TO, int DP>
hipError_t launch(const CacheAttnArgs& a, hipStream_t st) {
  const Cut c = cut_of(a);
  const dim3 grid(static_cast<unsigned>(c.slots ? c.pieces : a.B), a.cache.Hk * c.qtiles);
  {
    ProfScope prof("cache_attention", st);
    cache_attn_kernel<T, TO, DP><<<grid, 64 * kWaves, 0, st>>>(a, static_cast<int>(c.pieces), c.slots, c.fit, c.qtiles);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!c.slots) return hipSuccess;
  ProfScope prof("cache_join", st);
  cache_join_kernel<TO><<<dim3(static_cast<unsigned>(a.B * a.Hq)), 256, 0, st>>>(a, static_cast<int>(c.pieces));
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t launch_dim(const CacheAttnArgs& a, hipStream_t st) {
  if (a.cache.D <= 64) return launch<T, TO, 64>(a, st);
  return a.cache.D <= 128 ? launch<T, TO, 128>(a, st) : launch<T, TO, 256>(a, st);
}

}  // namespace

size_t cache_attn_workspace(const CacheAttnArgs& a) {
  const Cut c = cut_of(a);
  if (!c.slots) return 0;
  const size_t bytes = static_cast<size_t>(c.pieces) * a.Hq * (a.cache.D + 2) * sizeof(float) + a.B * sizeof(int2);
  return (bytes + 255) / 256 * 256;
}

hipError_t launch_cache_attn(const CacheAttnArgs& a, hipStream_t st) {
  if (a.bf16) return a.out_bf16 ? launch_dim<bf16_t, bf16_t>(a, st) : launch_dim<bf16_t, float>(a, st);
  return a.out_bf16 ? launch_dim<float, bf16_t>(a, st) : launch_dim<float, float>(a, st);
}

}  // namespace gdr
