// Rotary positions, and the append to a paged cache that applies them on the
// way.  Pair (a, b) of a head at angle w = pos freq:
//     (a, b) -> (a cos w - b sin w, b cos w + a sin w),   VJP: w -> -w.
// The angle is a product of 64 bits, reduced to half turns there: an fp32
// product is off by 2^-24 of the angle, a hundredth of a radian at position
// 131072.
//
// One workgroup takes `tokens` consecutive rows.  It first forms the cosines and
// sines of their pairs in LDS (once for all heads) and, for the append, each
// row's place in the cache; then it moves 16 channels a thread: eight pairs, or
// 16 channels that only move (those past R, and v).  Both ends of a pair are in
// one thread, so a call may work in place.
//
// Bound: memory, each row read and written once.  bf16, us (a graph of calls over
// rotating buffers): 16384 rows of 40 heads of 128, all turned, 64 (5.2 TB/s; a copy
// of 512 MiB reaches 6.2); 17 prompts of 17953 rows in all appended, 32 query and 8
// key heads, 88 (5.0 TB/s).  Rows of a workgroup: 8, 4, 2, 1 take 71, 67, 64, 63 and
// 100, 91, 88, 88.  Stores past the caches take 62 and 86, loads past them 61 and 92,
// but 2777 rows that are still in a cache then take 15-17 instead of 12, and what is
// stored is read next.

#include <algorithm>

#include "gdr_attn.h"
#include "gdr_device.h"

namespace gdr {
namespace {

constexpr int kMaxTokens = 2;    // rows of a workgroup
constexpr int kMaxPairs = 128;   // R / 2

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    float a[4], b[4];
    ld4<T>(p, a);
    ld4<T>(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      const b2 v{static_cast<__bf16>(x[2 * i]), static_cast<__bf16>(x[2 * i + 1])};
      w[i] = __builtin_bit_cast(uint32_t, v);
    }
    *reinterpret_cast<u32x4*>(p) = w;
  } else {
    const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
    st4<T>(p, a);
    st4<T>(p + 4, b);
  }
}

// The axis that pair i's position comes from.
__device__ __forceinline__ int pair_axis(const RotArgs& a, int i) {
  if (a.axes == 1) return 0;
  if (a.cycled) {
    const int x = i % a.axes;
    return i < a.axes * a.section[x] ? x : 0;
  }
  int x = 0, end = a.section[0];
  while (x < a.axes - 1 && i >= end) end += a.section[++x];
  return x;
}

// Rows row0 .. row0 + n - 1.
template <typename TI, typename TO>
__device__ __forceinline__ void rotary_rows(const RotArgs& a, int64_t row0, int n) {
  __shared__ float2 turn[kMaxTokens * kMaxPairs];
  __shared__ int64_t slot[kMaxTokens];  // a row's element offset in the cache; -1: none
  __shared__ int64_t place[kMaxTokens];
  __shared__ int live[kMaxTokens];
  const int tid = threadIdx.x, half = a.R / 2;

  if (a.append) {
    if (tid < kMaxTokens) live[tid] = 0, slot[tid] = -1;
    __syncthreads();
    // the sequence of each row, its place there, and the page's
    auto found = [&](int t, int64_t b, int64_t at) {
      place[t] = at;
      live[t] = 1;
      const CacheView& c = a.cache;
      const int64_t nth = at < 0 ? c.max_pages : at / c.page_size;
      if (nth >= c.max_pages) return;
      const int64_t page = c.table[b * c.table_row + nth];
      if (page < 0 || page >= c.pages) return;
      slot[t] = page * c.page_stride + (at - nth * c.page_size) * c.token_stride;
    };
    if (!a.cu) {
      if (tid < n) {
        const int64_t b = (row0 + tid) / a.T;
        found(tid, b, a.cache.lengths[b] - a.T + (row0 + tid - b * a.T));
      }
    } else {
      for (int64_t b = tid; b < a.B; b += 256) {
        const int64_t lo = a.cu[b], hi = a.cu[b + 1];
        const int64_t end = min(min(hi, lo + a.T) - row0, static_cast<int64_t>(n));
        for (int64_t t = max(lo - row0, int64_t(0)); t < end; ++t)
          found(static_cast<int>(t), b, a.cache.lengths[b] - hi + row0 + t);
      }
    }
    __syncthreads();
  }
  for (int u = tid; u < n * half; u += 256) {
    const int t = u / half, i = u - t * half;
    if (a.append && !live[t]) continue;
    const int64_t pos = a.pos ? a.pos[pair_axis(a, i) * a.rows + row0 + t] : place[t];
    double w = static_cast<double>(pos) * static_cast<double>(a.freq[i]) * 0.31830988618379067154;  // half turns
    w -= 2.0 * rint(0.5 * w);
    float s, c;
    sincospif(static_cast<float>(w), &s, &c);
    turn[t * half + i] = make_float2(c, a.back ? -s : s);
  }
  __syncthreads();

  const int per = a.D / 16, pairs = a.R / 16;
  const int heads = a.Hq + a.Hk + (a.append ? a.Hk : 0);
  const int units = heads * per;
  for (int u = tid; u < n * units; u += 256) {
    const int t = u / units, w = u - t * units;
    int h = w / per;
    const int x = w - h * per;
    if (a.append && !live[t]) continue;
    const int64_t row = row0 + t;
    const TI* src;
    TO* dst;
    bool turned = x < pairs;
    if (h < a.Hq) {
      src = static_cast<const TI*>(a.q) + row * a.q_row + h * a.D;
      dst = static_cast<TO*>(a.qo) + row * a.qo_row + h * a.D;
    } else {
      h -= a.Hq;
      const bool value = h >= a.Hk;
      if (value) h -= a.Hk, turned = false;
      src = value ? static_cast<const TI*>(a.v) + row * a.v_row : static_cast<const TI*>(a.k) + row * a.k_row;
      src += h * a.D;
      if (a.append) {
        if (slot[t] < 0) continue;
        dst = static_cast<TO*>(value ? a.vc : a.ko) + slot[t] + h * a.cache.head_stride;
      } else {
        dst = static_cast<TO*>(a.ko) + row * a.ko_row + h * a.D;
      }
    }
    float lo[8], hi[8];
    // a thread's two runs of 8: the ends of its pairs, or neighbours
    const bool split = turned && !a.adjacent;
    const int at = split ? 8 * x : 16 * x, to = split ? half + 8 * x : 16 * x + 8;
    load8<TI>(src + at, lo);
    load8<TI>(src + to, hi);
    if (turned) {
      const float2* cs = turn + t * half + 8 * x;
      if (split) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = cs[i];
          const float p = lo[i], r = hi[i];
          lo[i] = p * f.x - r * f.y;
          hi[i] = r * f.x + p * f.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = cs[i], g = cs[4 + i];
          const float p = lo[2 * i], r = lo[2 * i + 1], s = hi[2 * i], z = hi[2 * i + 1];
          lo[2 * i] = p * f.x - r * f.y;
          lo[2 * i + 1] = r * f.x + p * f.y;
          hi[2 * i] = s * g.x - z * g.y;
          hi[2 * i + 1] = z * g.x + s * g.y;
        }
      }
    }
    store8<TO>(dst + at, lo);
    store8<TO>(dst + to, hi);
  }
}

template <typename TI, typename TO>
__global__ __launch_bounds__(256) void rotary_kernel(RotArgs a, int tokens) {
  const int64_t step = static_cast<int64_t>(gridDim.x) * tokens;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * tokens; row0 < a.rows; row0 += step) {
    rotary_rows<TI, TO>(a, row0, static_cast<int>(min(static_cast<int64_t>(tokens), a.rows - row0)));
    __syncthreads();  // the rows' turns and places are read
  }
}

template <typename TI, typename TO>
hipError_t launch(const RotArgs& a, hipStream_t st) {
  // a step of single tokens spreads over the card, many rows share a workgroup
  const int64_t most = (a.rows + 1023) / 1024;
  const int tokens = static_cast<int>(most < kMaxTokens ? (most < 1 ? 1 : most) : kMaxTokens);
  // a launch has less than 2^32 threads
  const int64_t blocks = std::min<int64_t>((a.rows + tokens - 1) / tokens, 1 << 22);
  rotary_kernel<TI, TO><<<dim3(static_cast<unsigned>(blocks)), 256, 0, st>>>(a, tokens);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotary(const RotArgs& a, hipStream_t st) {
  ProfScope prof(a.append ? "cache_append" : "rotary", st);
  if (a.io_bf16) return a.out_bf16 ? launch<bf16_t, bf16_t>(a, st) : launch<bf16_t, float>(a, st);
  return a.out_bf16 ? launch<float, bf16_t>(a, st) : launch<float, float>(a, st);
}

}  // namespace gdr
