// Group norm over the last axis of [rows, G, D], with an affine map and an
// activation, and its VJP.  Per row and group, in fp32:
//     n = (x - mean) r,  r = (mean (x - mean)^2 + eps)^(-1/2)   (mean: 0 without GDR_NORM_CENTER)
//     u = w n + b,  y = u silu(z) | silu(u) | u
//     du = dy silu(z),  dz = dy u silu'(z);  or du = dy silu'(u);  or du = dy
//     dn = w du,  dx = r (dn - mean dn - n mean(dn n))   (mean dn: only when centred)
//     dw = sum over rows of du n,  db = sum over rows of du.
//
// Layout.  A group is held by LPG lanes (the power of two at or above D / 8),
// 8 channels each, so x, z, dy and the results move once, in 16-byte
// accesses, and both statistics come from registers (the variance from the
// centred values, a second pass that costs no memory).  A slot of LPG lanes
// keeps one group index for all the rows it walks, so weights are read once
// and the weights' gradients are summed in its registers.  Bound: memory; 16384
// rows of 32 x 128, bf16, with a gate: forward 80 us (5.04 TB/s), VJP 136 (4.92
// TB/s); back to back 71 and 128; a copy of 512 MiB reaches 6.2 TB/s.

#include <algorithm>

#include "gdr_device.h"
#include "gdr_norm.h"

namespace gdr {
namespace {

constexpr int kPer = 8;  // channels per lane

// bf16 rows move past the caches (non-temporal): each is touched once.  16384
// rows of 32 x 128, rotating: forward 88 -> 82 us, VJP 147 -> 139.
typedef uint32_t u32x4n __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ void ld8(const T* p, float (&x)[8]) {
  float a[4], b[4];
  if constexpr (sizeof(T) == 2) {
    const u32x4n w = __builtin_nontemporal_load(reinterpret_cast<const u32x4n*>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    ld4<T>(p, a);
    ld4<T>(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
  }
}

template <typename T> __device__ __forceinline__ void st8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      typedef __bf16 b2 __attribute__((ext_vector_type(2)));
      const b2 v{static_cast<__bf16>(x[2 * i]), static_cast<__bf16>(x[2 * i + 1])};
      w[i] = __builtin_bit_cast(uint32_t, v);
    }
    __builtin_nontemporal_store(u32x4n{w[0], w[1], w[2], w[3]}, reinterpret_cast<u32x4n*>(p));
  } else {
    const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
    st4<T>(p, a);
    st4<T>(p + 4, b);
  }
}

template <int LPG>
__device__ __forceinline__ float group_sum(float x) {
  if constexpr (LPG == 8 || LPG == 16) return group_sum_dpp<LPG>(x);
  else if constexpr (LPG == 64) return rows4_sum(group_sum_dpp<16>(x));
  else if constexpr (LPG == 32) { x = group_sum_dpp<16>(x); return x + __shfl_xor(x, 16, 64); }
  else return xsum<1, LPG>(x);
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + __expf(-x)); }

// Where a lane works: its slot's group, its first row, and its channels.
struct NormPos {
  int g, c, ch;      // group, first channel in the group, first channel of the row
  int64_t row;
  bool on;           // the lane has channels
};
template <int LPG>
__device__ __forceinline__ NormPos norm_pos(const NormArgs& a, int phases) {
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * (256 / LPG) + threadIdx.x / LPG;
  NormPos p;
  p.g = static_cast<int>(slot % a.G);
  p.row = slot / a.G;
  p.c = threadIdx.x % LPG * kPer;
  p.ch = p.g * a.D + p.c;
  p.on = p.c < a.D && p.row < phases;
  if (p.row >= phases) p.row = a.rows;  // a slot past the last: no rows
  return p;
}

__device__ __forceinline__ void load_params(const NormArgs& a, const NormPos& p, float (&w)[8], float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f, b[i] = 0.f;
  const int at = a.shared ? p.c : p.ch;
  if (p.on && a.w) ld8<float>(a.w + at, w);
  if (p.on && a.b) ld8<float>(a.b + at, b);
}

// Centres x in place (lanes without channels keep zeros) and gives r.
template <int LPG>
__device__ __forceinline__ float norm_stats(const NormArgs& a, const NormPos& p, float (&x)[8]) {
  const float inv = 1.f / a.D;
  if (a.center) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i];
    const float mu = group_sum<LPG>(s) * inv;
    if (p.on)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] -= mu;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += x[i] * x[i];
  return 1.f / sqrtf(group_sum<LPG>(s) * inv + a.eps);
}

template <typename TI, typename TO, int LPG>
__global__ __launch_bounds__(256) void norm_fwd_kernel(NormArgs a, int phases) {
  const NormPos p = norm_pos<LPG>(a, phases);
  float w[8], b[8];
  load_params(a, p, w, b);
  for (int64_t row = p.row; row < a.rows; row += phases) {
    float x[8] = {}, z[8] = {}, y[8];
    if (p.on) {
      ld8<TI>(static_cast<const TI*>(a.x) + row * a.x_row + p.ch, x);
      if (a.z) ld8<TI>(static_cast<const TI*>(a.z) + row * a.z_row + p.ch, z);
    }
    const float r = norm_stats<LPG>(a, p, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float u = w[i] * (x[i] * r) + b[i];
      y[i] = a.z ? u * (z[i] * sigmoid(z[i])) : a.silu ? u * sigmoid(u) : u;
    }
    if (p.on) st8<TO>(static_cast<TO*>(a.y) + row * (static_cast<int64_t>(a.G) * a.D) + p.ch, y);
  }
}

// part: [phases][2][G * D] sums of du n and du over the slot's rows; with a
// shared weight the slots of a block are added first: [blocks][2][D].
template <typename TI, typename TO, int LPG>
__global__ __launch_bounds__(256) void norm_bwd_kernel(NormArgs a, int phases) {
  const NormPos p = norm_pos<LPG>(a, phases);
  const int64_t C = static_cast<int64_t>(a.G) * a.D;
  float w[8], b[8], dw[8] = {}, db[8] = {};
  load_params(a, p, w, b);
  const float inv = 1.f / a.D;
  for (int64_t row = p.row; row < a.rows; row += phases) {
    float x[8] = {}, z[8] = {}, dy[8] = {}, dx[8], dz[8];
    if (p.on) {
      ld8<TI>(static_cast<const TI*>(a.x) + row * a.x_row + p.ch, x);
      ld8<TI>(static_cast<const TI*>(a.dy) + row * C + p.ch, dy);
      if (a.z) ld8<TI>(static_cast<const TI*>(a.z) + row * a.z_row + p.ch, z);
    }
    const float r = norm_stats<LPG>(a, p, x);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = x[i] * r, u = w[i] * n + b[i];
      float du = dy[i];
      if (a.z) {
        const float sg = sigmoid(z[i]);
        dz[i] = dy[i] * u * (sg * (1.f + z[i] * (1.f - sg)));
        du = dy[i] * (z[i] * sg);
      } else if (a.silu) {
        const float sg = sigmoid(u);
        du = dy[i] * (sg * (1.f + u * (1.f - sg)));
      }
      dw[i] += du * n;
      db[i] += du;
      const float dn = du * w[i];
      x[i] = n;
      dx[i] = dn;
      s1 += dn;
      s2 += dn * n;
    }
    s2 = group_sum<LPG>(s2) * inv;
    s1 = a.center ? group_sum<LPG>(s1) * inv : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) dx[i] = r * (dx[i] - s1 - x[i] * s2);
    if (p.on) {
      st8<TO>(static_cast<TO*>(a.dx) + row * C + p.ch, dx);
      if (a.z) st8<TO>(static_cast<TO*>(a.dz) + row * C + p.ch, dz);
    }
  }
  if (!a.dw && !a.db) return;
  if (!a.shared) {
    const int64_t phase = (static_cast<int64_t>(blockIdx.x) * (256 / LPG) + threadIdx.x / LPG) / a.G;
    if (p.on) {
      float* at = a.part + phase * 2 * C + p.ch;
      if (a.dw) st8<float>(at, dw);
      if (a.db) st8<float>(at + C, db);
    }
    return;
  }
  __shared__ float sum[256][kPer + 1];
  for (int which = 0; which < 2; ++which) {
    if (which ? !a.db : !a.dw) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[threadIdx.x][i] = which ? db[i] : dw[i];
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += 256) {
      float s = 0.f;
      for (int k = 0; k < 256 / LPG; ++k) s += sum[k * LPG + c / kPer][c % kPer];
      a.part[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.D + c] = s;
    }
  }
}

// dw, db: column sums of the n partial rows, in a fixed order: 64 row lanes
// per 16 columns, each over every 64th row, then the 64 eight at a time (64
// bits).  Bound: latency; eight rows are in flight at a time.
__global__ __launch_bounds__(1024) void norm_params_kernel(const float* part, float* dw, float* db, int64_t n,
                                                           int C) {
  __shared__ double sum[64][17];
  const int col = threadIdx.x & 15, lane = threadIdx.x >> 4, c = blockIdx.x * 16 + col;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  double s = 0.0;
  if (c < C)
    for (int64_t i = lane; i < n; i += 512) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = i + 64 * u < n ? part[((i + 64 * u) * 2 + blockIdx.y) * C + c] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
  sum[lane][col] = s;
  __syncthreads();
  if (lane < 8) {
    s = 0.0;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += sum[8 * lane + k][col];
  }
  __syncthreads();
  if (lane < 8) sum[lane][col] = s;
  __syncthreads();
  if (lane == 0 && c < C) {
#pragma unroll
    for (int k = 1; k < 8; ++k) s += sum[k][col];
    out[c] = static_cast<float>(s);
  }
}

int lanes_per_group(int D) {
  int l = 1;
  while (l * kPer < D) l *= 2;
  return l;
}

// Row phases of a launch: one slot per group and phase.  Enough slots for
// `waves` waves on each of the 256 CUs, and no more phases than rows.
int norm_phases(const NormArgs& a, int waves) {
  const int64_t slots = 256ll * waves * (64 / lanes_per_group(a.D));
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.rows, slots / a.G)));
}
int64_t norm_blocks(const NormArgs& a, int phases) {
  const int64_t per = 256 / lanes_per_group(a.D);
  return (static_cast<int64_t>(phases) * a.G + per - 1) / per;
}
// The forward keeps nothing per slot, and more waves than fit hide its loads;
// the VJP writes a partial row per phase.  16384 rows of 32 x 128: forward 86,
// 82, 80 us at 16, 32, 64 waves; VJP 148, 136, 139 at 8, 12, 16, and 1237 rows
// 15.6, 15.3, 16.8.
constexpr int kFwdWaves = 64, kBwdWaves = 12;

template <typename TI, typename TO>
hipError_t launch_fwd(const NormArgs& a, hipStream_t st) {
  const int phases = norm_phases(a, kFwdWaves);
  const dim3 grid(static_cast<unsigned>(norm_blocks(a, phases)));
  switch (lanes_per_group(a.D)) {
    case 1: norm_fwd_kernel<TI, TO, 1><<<grid, 256, 0, st>>>(a, phases); break;
    case 2: norm_fwd_kernel<TI, TO, 2><<<grid, 256, 0, st>>>(a, phases); break;
    case 4: norm_fwd_kernel<TI, TO, 4><<<grid, 256, 0, st>>>(a, phases); break;
    case 8: norm_fwd_kernel<TI, TO, 8><<<grid, 256, 0, st>>>(a, phases); break;
    case 16: norm_fwd_kernel<TI, TO, 16><<<grid, 256, 0, st>>>(a, phases); break;
    case 32: norm_fwd_kernel<TI, TO, 32><<<grid, 256, 0, st>>>(a, phases); break;
    default: norm_fwd_kernel<TI, TO, 64><<<grid, 256, 0, st>>>(a, phases); break;
  }
  return hipGetLastError();
}

template <typename TI, typename TO>
hipError_t launch_bwd(const NormArgs& a, hipStream_t st) {
  const int phases = norm_phases(a, kBwdWaves);
  const int64_t blocks = norm_blocks(a, phases);
  const dim3 grid(static_cast<unsigned>(blocks));
  {
    ProfScope prof("norm_bwd", st);
    switch (lanes_per_group(a.D)) {
      case 1: norm_bwd_kernel<TI, TO, 1><<<grid, 256, 0, st>>>(a, phases); break;
      case 2: norm_bwd_kernel<TI, TO, 2><<<grid, 256, 0, st>>>(a, phases); break;
      case 4: norm_bwd_kernel<TI, TO, 4><<<grid, 256, 0, st>>>(a, phases); break;
      case 8: norm_bwd_kernel<TI, TO, 8><<<grid, 256, 0, st>>>(a, phases); break;
      case 16: norm_bwd_kernel<TI, TO, 16><<<grid, 256, 0, st>>>(a, phases); break;
      case 32: norm_bwd_kernel<TI, TO, 32><<<grid, 256, 0, st>>>(a, phases); break;
      default: norm_bwd_kernel<TI, TO, 64><<<grid, 256, 0, st>>>(a, phases); break;
    }
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!a.dw && !a.db) return hipSuccess;
  ProfScope prof("norm_params", st);
  const int C = a.shared ? a.D : a.G * a.D;
  norm_params_kernel<<<dim3((C + 15) / 16, 2), 1024, 0, st>>>(a.part, a.dw, a.db, a.shared ? blocks : phases, C);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st) {
  ProfScope prof("norm_fwd", st);
  if (a.io_bf16) return a.out_bf16 ? launch_fwd<bf16_t, bf16_t>(a, st) : launch_fwd<bf16_t, float>(a, st);
  return a.out_bf16 ? launch_fwd<float, bf16_t>(a, st) : launch_fwd<float, float>(a, st);
}

size_t norm_bwd_workspace(const NormArgs& a) {
  const int phases = norm_phases(a, kBwdWaves);
  const size_t n = a.shared ? static_cast<size_t>(norm_blocks(a, phases)) * a.D
                            : static_cast<size_t>(phases) * a.G * a.D;
  return (n * 2 * sizeof(float) + 255) / 256 * 256;
}

hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st) {
  if (a.io_bf16) return a.out_bf16 ? launch_bwd<bf16_t, bf16_t>(a, st) : launch_bwd<bf16_t, float>(a, st);
  return a.out_bf16 ? launch_bwd<float, bf16_t>(a, st) : launch_bwd<float, float>(a, st);
}

}  // namespace gdr
