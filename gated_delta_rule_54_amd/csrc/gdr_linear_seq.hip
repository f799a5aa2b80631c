// Linear attention with a decay for each head, token by token: single tokens,
// short sequences, and every shape in fp32 arithmetic.  Also the last step of
// the VJP, which both algorithms share: head sums and the decay's gradient.

#include <type_traits>

#include "gdr_device.h"
#include "gdr_linear.h"

namespace gdr {
namespace {

typedef float f32x4n __attribute__((ext_vector_type(4)));

// One token as one thread sees it: its R rows of x and y, its 4 columns of z.
template <int R>
struct LinTok {
  float x[R], y[R], z[4], ex[4], g;
};

template <typename TI, int R>
__device__ __forceinline__ void lin_load(LinTok<R>& k, const LinChain& c, const float* g, int64_t gstep, int64_t row,
                                         int h, int r0, int col) {
  const TI* x = static_cast<const TI*>(c.x) + row * c.xr + static_cast<int64_t>(h / c.xg) * c.D1;
  const TI* y = static_cast<const TI*>(c.y) + row * c.yr + static_cast<int64_t>(h / c.yg) * c.D1;
  const TI* z = static_cast<const TI*>(c.z) + row * c.zr + static_cast<int64_t>(h / c.zg) * c.D2;
#pragma unroll
  for (int m = 0; m < R; m += 4) {
    float tx[4] = {0.f, 0.f, 0.f, 0.f}, ty[4] = {0.f, 0.f, 0.f, 0.f};
    if (r0 + m < c.D1) {
      ld4<TI>(x + r0 + m, tx);
      ld4<TI>(y + r0 + m, ty);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) k.x[m + i] = tx[i], k.y[m + i] = ty[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) k.z[i] = 0.f, k.ex[i] = 0.f;
  if (col < c.D2) {
    ld4<TI>(z + col, k.z);
    if (c.ex)
      ld4<TI>(static_cast<const TI*>(c.ex) + row * c.er + static_cast<int64_t>(h / c.eg) * c.D2 + col, k.ex);
  }
  k.g = g ? g[row * gstep + h] : 0.f;
}

// A workgroup owns all D1 rows of one state slice of 64 columns: thread
// (rg, cg) holds rows R rg .. R rg + R - 1 of columns 4 cg .. 4 cg + 3 in
// registers for the whole sequence.  Per token the state is updated and the
// output's partial sums are reduced over the 16 row groups: across a wave's
// four by row swaps, across the four waves through LDS (one barrier a token,
// the buffers alternate).  Bound: at one token a call, the state's read and
// write; over a sequence, the barrier and the load latency of each token.
template <typename TI, int R>
__global__ __launch_bounds__(256) void lin_seq_kernel(LinChains a) {
  __shared__ float red[2][4][kLinSlice];
  int64_t blk = blockIdx.x;
  int ci = 0;
  const int64_t heads = a.B * a.Hv;
  if (a.n > 1 && blk >= heads * lin_slices(a.c[0].D2)) {
    blk -= heads * lin_slices(a.c[0].D2), ci = 1;
    if (blk >= heads * lin_slices(a.c[1].D2)) blk -= heads * lin_slices(a.c[1].D2), ci = 2;
  }
  const LinChain c = lin_chain(ci);
  const int nsl = lin_slices(c.D2), sl = static_cast<int>(blk % nsl);
  const int64_t bh = blk / nsl;
  const int h = static_cast<int>(bh % a.Hv);
  const int64_t b = bh / a.Hv;
  const int tid = threadIdx.x, cg = tid & 15, rg = tid >> 4, wave = tid >> 6;
  const int r0 = rg * R, col = sl * kLinSlice + 4 * cg;
  const LinSpan sp = lin_span(a.cu, b, a.T);
  const int64_t st0 = bh * c.D1 * c.D2;

  float H[R][4];
#pragma unroll
  for (int m = 0; m < R; ++m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) H[m][i] = 0.f;
    if (c.s_in && r0 + m < c.D1 && col < c.D2) {
      const float* p = c.s_in + st0 + static_cast<int64_t>(r0 + m) * c.s1 + static_cast<int64_t>(col) * c.s2;
      if (c.s2 == 1) {
        const f32x4n x = __builtin_nontemporal_load(reinterpret_cast<const f32x4n*>(p));
#pragma unroll
        for (int i = 0; i < 4; ++i) H[m][i] = x[i];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) H[m][i] = p[i * c.s2];
      }
    }
  }

  const int64_t gstep = a.head_decay ? 0 : a.Hv;
  LinTok<R> k, nx;
  if (sp.len > 0) lin_load<TI, R>(k, c, a.g, gstep, sp.t0 + (c.rev ? sp.len - 1 : 0), h, r0, col);
  float before = 1.f;  // backward in time: the factor of the token after this one
  for (int64_t i = 0; i < sp.len; ++i) {
    const int64_t t = c.rev ? sp.len - 1 - i : i;
    if (i + 1 < sp.len) lin_load<TI, R>(nx, c, a.g, gstep, sp.t0 + (c.rev ? t - 1 : t + 1), h, r0, col);
    const float al = expf(k.g), f = c.rev ? before : al;
    before = al;
    float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        H[m][j] = f * H[m][j] + k.y[m] * k.z[j];
        o[j] += k.x[m] * H[m][j];
      }
    if (c.out) {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = rows4_sum(o[j]);
      float(&buf)[4][kLinSlice] = red[i & 1];
      if ((tid & 63) < 16) *reinterpret_cast<float4*>(&buf[wave][4 * cg]) = make_float4(o[0], o[1], o[2], o[3]);
      __syncthreads();
      if (tid < 16) {
        float s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          s[j] = (buf[0][4 * cg + j] + buf[1][4 * cg + j]) + (buf[2][4 * cg + j] + buf[3][4 * cg + j]);
        if (col < c.D2) {
          const int64_t row = c.out_partial ? lin_part_row(a, b, sp, t) : sp.t0 + t;
          const int64_t at = (row * a.Hv + h) * c.D2 + col;
          if (c.out_partial || !a.out_bf16) st4<float>(static_cast<float*>(c.out) + at, s);
          else st4<bf16_t>(static_cast<bf16_t*>(c.out) + at, s);
        }
        if (c.ex) {
          const float e = row16_sum(s[0] * k.ex[0] + s[1] * k.ex[1] + s[2] * k.ex[2] + s[3] * k.ex[3]);
          if (tid == 0) c.e[(static_cast<int64_t>(sl) * a.Hv + h) * a.rows + lin_part_row(a, b, sp, t)] = e;
        }
      }
    }
    k = nx;
  }

  if (c.xdot) {
    float s = 0.f;
    if (c.dot && col < c.D2) {
      const float* p = c.dot + st0 + static_cast<int64_t>(col) * c.s2;
#pragma unroll
      for (int m = 0; m < R; ++m)
        if (r0 + m < c.D1)
#pragma unroll
          for (int i = 0; i < 4; ++i) s += H[m][i] * p[static_cast<int64_t>(r0 + m) * c.s1 + i * c.s2];
    }
    s = rows4_sum(row16_sum(s));
    __syncthreads();
    if ((tid & 63) == 0) red[0][wave][0] = s;
    __syncthreads();
    if (tid == 0) c.xdot[bh * nsl + sl] = (red[0][0][0] + red[0][1][0]) + (red[0][2][0] + red[0][3][0]);
  }
  if (c.s_out && col < c.D2) {
    const float f = c.rev ? before : 1.f;
#pragma unroll
    for (int m = 0; m < R; ++m)
      if (r0 + m < c.D1) {
        float* p = c.s_out + st0 + static_cast<int64_t>(r0 + m) * c.s1 + static_cast<int64_t>(col) * c.s2;
        const float v[4] = {f * H[m][0], f * H[m][1], f * H[m][2], f * H[m][3]};
        if (c.s2 == 1) {
          __builtin_nontemporal_store(f32x4n{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4n*>(p));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i * c.s2] = v[i];
        }
      }
  }
}

// One token forward.  A workgroup owns all rows of kLinSlice columns of a head's
// state and passes over them 256 x 4 elements at a time: a wave reads and writes
// rows that follow each other, where the kernel above, whose threads hold rows
// of their own, touches four places 4 KB apart.  The state is touched once, so
// past the caches (non-temporal).  The output's sums over the workgroup's row
// groups meet in LDS.  Bound: the state's read and write.  Measured, 32 heads of
// 128 x 128, states rotating: 256 sequences 186 us (5.75 TB/s; the kernel above
// 288), 64 sequences 50 (72), 8 sequences 8.7 (10.5).  Slices of 32 columns take
// 198, 52 and 10.0, of 128 columns 196, 51 and 10.2.
template <typename TI>
__global__ __launch_bounds__(256) void lin_token_kernel(LinChains a) {
  __shared__ float kx[256], qx[256];  // D1 <= 256
  __shared__ float4 red[256];
  const LinChain c = lin_chain(0);
  const int nsl = lin_slices(c.D2), col0 = static_cast<int>(blockIdx.x % nsl) * kLinSlice;
  const int64_t bh = blockIdx.x / nsl, b = bh / a.Hv;
  const int h = static_cast<int>(bh % a.Hv), tid = threadIdx.x;
  const int nc = min(kLinSlice, c.D2 - col0) / 4, step = 256 / nc, cg = tid % nc, rg = tid / nc;
  const LinSpan sp = lin_span(a.cu, b, a.T);
  const int64_t row = sp.t0;
  const bool any = sp.len > 0, on = rg < step;
  float z[4] = {0.f, 0.f, 0.f, 0.f}, f = 1.f;
  if (any) {
    const TI* x = static_cast<const TI*>(c.x) + row * c.xr + static_cast<int64_t>(h / c.xg) * c.D1;
    const TI* y = static_cast<const TI*>(c.y) + row * c.yr + static_cast<int64_t>(h / c.yg) * c.D1;
    for (int i = tid; i < c.D1; i += 256) qx[i] = ld1(x + i), kx[i] = ld1(y + i);
    ld4<TI>(static_cast<const TI*>(c.z) + row * c.zr + static_cast<int64_t>(h / c.zg) * c.D2 + col0 + 4 * cg, z);
    if (a.g) f = expf(a.g[a.head_decay ? h : row * a.Hv + h]);
  }
  __syncthreads();
  const int64_t at = bh * c.D1 * c.D2 + col0 + 4 * cg;
  const float* in = c.s_in ? c.s_in + at : nullptr;
  float* out = c.s_out ? c.s_out + at : nullptr;
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;
  for (int r = on ? rg : c.D1; r < c.D1; r += U * step) {
    f32x4n H[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      H[u] = f32x4n{0.f, 0.f, 0.f, 0.f};
      const int i = r + u * step;
      if (in && i < c.D1)
        H[u] = __builtin_nontemporal_load(reinterpret_cast<const f32x4n*>(in + static_cast<int64_t>(i) * c.D2));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = r + u * step;
      if (i < c.D1) {
        if (any) {
          const float y = kx[i], x = qx[i];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            H[u][j] = f * H[u][j] + y * z[j];
            o[j] += x * H[u][j];
          }
        }
        if (out) __builtin_nontemporal_store(H[u], reinterpret_cast<f32x4n*>(out + static_cast<int64_t>(i) * c.D2));
      }
    }
  }
  if (!any) return;
  red[tid] = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  if (tid < 4 * nc) {
    const float* p = reinterpret_cast<const float*>(red) + tid;
    float s = 0.f;
    for (int i = 0; i < step; ++i) s += p[4 * nc * i];
    const int64_t to = (row * a.Hv + h) * c.D2 + col0 + tid;
    if (a.out_bf16) st1(static_cast<bf16_t*>(c.out) + to, s);
    else st1(static_cast<float*>(c.out) + to, s);
  }
}

// The sequence that holds row r of a ragged batch: the last one that starts at
// or before it.
__device__ __forceinline__ int64_t lin_sequence_of(const int64_t* cu, int64_t B, int64_t r) {
  int64_t lo = 0, hi = B;
  while (hi - lo > 1) {
    const int64_t m = (lo + hi) / 2;
    if (cu[m] <= r) lo = m;
    else hi = m;
  }
  return lo;
}

// Sums fp32 partial rows [n][Hv][Dk] over the value heads of each key head into
// rows [..][Hk][Dk] of TO; blockIdx.y: dq, dk.  One thread per 4 columns.
template <typename TO>
__global__ __launch_bounds__(256) void lin_group_sum_kernel(const float* pdq, const float* pdk, TO* dq, TO* dk,
                                                            int64_t B, int64_t T, int64_t n, bool packed, int Hk,
                                                            int Hv, int Dk, const int64_t* cu) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int per = Hk * (Dk / 4);
  const int64_t r = i / per;
  if (r >= n) return;
  const int u = static_cast<int>(i % per), hk = u / (Dk / 4), d = u % (Dk / 4) * 4;
  const int64_t b = cu && packed ? lin_sequence_of(cu, B, r) : r / T;
  const LinSpan sp = lin_span(cu, b, T);
  const int64_t t = packed ? r - sp.t0 : r % T;
  if (t < 0 || t >= sp.len) return;
  const int G = Hv / Hk;
  const float* p = (blockIdx.y ? pdk : pdq) + (r * Hv + hk * G) * Dk + d;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < G; ++j) {
    float x[4];
    ld4<float>(p + static_cast<int64_t>(j) * Dk, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += x[e];
  }
  st4<TO>((blockIdx.y ? dk : dq) + ((sp.t0 + t) * Hk + hk) * Dk + d, s);
}

// dg of one segment of one sequence and value head: the suffix sums of
// e_q - e_k from the segment's end, on top of <S, dS> there.  The sums run in
// 64 bits: they telescope to what the later tokens of the segment give, so
// their terms cancel.  One workgroup walks its segment from the end, 1024
// tokens at a time: a step is a chain of latencies (loads, shuffles, two
// barriers), so long ones are worth their idle lanes in short segments.  Where
// the factor is zero the state before has no part in anything after it: dg is 0,
// not what the sums' roundings leave.
constexpr float kNoFactor = -104.f;  // e^g below half of fp32's least value
constexpr int kDgStep = 1024;
__global__ __launch_bounds__(kDgStep) void lin_dg_kernel(const float* eq, const float* ek, const float* xdot, int nsl,
                                                         int dots, const float* g, float* dg, double* dgsum, int64_t B, int64_t T,
                                                         int64_t rows, bool packed, int Hv, int64_t segments,
                                                         int64_t seg, const int64_t* cu) {
  constexpr int W = kDgStep / 64;
  __shared__ double wsum[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t s = blockIdx.x % segments, bh = blockIdx.x / segments, b = bh / Hv;
  const int h = static_cast<int>(bh % Hv);
  const LinSpan sp = lin_span(cu, b, T);
  const int64_t t0 = s * seg, t1 = sp.len < t0 + seg ? sp.len : t0 + seg;
  double carry = 0.0, total = 0.0;
  for (int j = 0; j < dots; ++j) carry += xdot[(s * B * Hv + bh) * dots + j];
  const int64_t row0 = packed ? sp.t0 : b * T;
  auto term = [&](int64_t t) {
    double v = 0.0;
    if (t >= t0)
      for (int j = 0; j < nsl; ++j) {
        const int64_t at = (static_cast<int64_t>(j) * Hv + h) * rows + row0 + t;
        v += static_cast<double>(eq[at]) - static_cast<double>(ek[at]);
      }
    return v;
  };
  double next = term(t1 - 1 - tid);
  for (int64_t end = t1; end > t0; end -= kDgStep) {
    const int64_t t = end - 1 - tid;
    double p = next;
    next = term(t - kDgStep);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double q = __shfl_up(p, m, 64);
      if (lane >= m) p += q;
    }
    if (lane == 63) wsum[wave] = p;
    __syncthreads();
    double base = carry, all = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < wave) base += wsum[w];
      all += wsum[w];
    }
    __syncthreads();
    carry += all;
    p += base;
    if (t >= t0) {
      if (dgsum) total += p;
      else {
        const int64_t at = (sp.t0 + t) * Hv + h;
        dg[at] = g[at] < kNoFactor ? 0.f : static_cast<float>(p);
      }
    }
  }
  if (dgsum) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) total += __shfl_xor(total, m, 64);
    if (lane == 0) wsum[wave] = total;
    __syncthreads();
    if (tid == 0) {
      double all = 0.0;
      for (int w = 0; w < W; ++w) all += wsum[w];
      dgsum[(b * segments + s) * Hv + h] = all;
    }
  }
}

// dg [Hv] with a decay per head: the segments' sums, one wave per head.
__global__ __launch_bounds__(64) void lin_dg_head_kernel(const double* dgsum, const float* g, float* dg, int64_t n,
                                                         int Hv) {
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 64) s += dgsum[i * Hv + h];
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
  if (threadIdx.x == 0) dg[h] = g[h] < kNoFactor ? 0.f : static_cast<float>(s);
}

__global__ __launch_bounds__(256) void lin_zero_kernel(float* p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

template <typename TI>
hipError_t seq_launch(const LinChains& a, int rows, int64_t blocks, hipStream_t st) {
  ProfScope prof("linear_seq", st);
  const dim3 grid(static_cast<unsigned>(blocks));
  if (rows <= 64) lin_seq_kernel<TI, 4><<<grid, 256, 0, st>>>(a);
  else if (rows <= 128) lin_seq_kernel<TI, 8><<<grid, 256, 0, st>>>(a);
  else lin_seq_kernel<TI, 16><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

LinChains lin_forward_chains(const LinShape& s, const LinFwdArgs& a) {
  LinChains L{};
  const int G = s.Hv / s.Hk;
  L.n = 1, L.segments = 1, L.seg = s.T;
  L.B = s.B, L.T = s.T, L.rows = s.rows, L.packed = s.packed, L.Hv = s.Hv, L.group = G, L.g = a.g, L.head_decay = s.head_decay;
  L.out_bf16 = s.out_bf16, L.cu = a.cu;
  LinChain& c = L.c[0];
  c.x = a.q, c.xr = s.q_row, c.xg = G;
  c.y = a.k, c.yr = s.k_row, c.yg = G;
  c.z = a.v, c.zr = s.v_row, c.zg = 1;
  c.D1 = s.Dk, c.D2 = s.Dv;
  c.s_in = a.h0, c.s_out = a.ht, c.s1 = s.Dv, c.s2 = 1;
  c.out = a.o;
  return L;
}

size_t lin_bwd_parts(const LinShape& s, int64_t segments, bool summed, char* base, LinBwdParts* p) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* at = base ? base + off : nullptr;  // null: sizes only
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t bh = static_cast<size_t>(s.B) * s.Hv, n = static_cast<size_t>(s.Hv) * s.rows, nsl = lin_slices(s.Dk);
  p->eq = reinterpret_cast<float*>(take(2 * nsl * n * 4));
  p->ek = reinterpret_cast<float*>(take(2 * nsl * n * 4));
  p->xdot = reinterpret_cast<float*>(take(segments * bh * nsl * 4 * 4));
  const size_t heads = s.Hv == s.Hk ? 0 : summed ? s.Hk : s.Hv, part = heads * s.rows * s.Dk * 4;
  p->pdq = reinterpret_cast<float*>(take(part));
  p->pdk = reinterpret_cast<float*>(take(part));
  p->dgsum = reinterpret_cast<double*>(take(s.head_decay ? segments * bh * 8 : 0));
  return off;
}

LinChains lin_backward_chains(const LinShape& s, const LinBwdArgs& a, const LinBwdParts& p) {
  LinChains L{};
  const int G = s.Hv / s.Hk;
  const int64_t d_row = static_cast<int64_t>(s.Hv) * s.Dv;
  L.n = 3, L.segments = 1, L.seg = s.T;
  L.B = s.B, L.T = s.T, L.rows = s.rows, L.packed = s.packed, L.Hv = s.Hv, L.group = G, L.g = a.g, L.head_decay = s.head_decay;
  L.out_bf16 = s.out_bf16, L.cu = a.cu;
  LinChain& q = L.c[0];  // dq
  q.x = a.dout, q.xr = d_row, q.xg = 1;
  q.y = a.v, q.yr = s.v_row, q.yg = 1;
  q.z = a.k, q.zr = s.k_row, q.zg = G;
  q.D1 = s.Dv, q.D2 = s.Dk;
  q.s_in = a.h0, q.s1 = 1, q.s2 = s.Dv;
  q.out = G > 1 ? p.pdq : a.dq, q.out_partial = G > 1;
  if (a.dg) {
    q.ex = a.q, q.er = s.q_row, q.eg = G, q.e = p.eq;
    q.dot = a.dht, q.xdot = p.xdot;
  }
  LinChain& k = L.c[1];  // dk
  k.x = a.v, k.xr = s.v_row, k.xg = 1;
  k.y = a.dout, k.yr = d_row, k.yg = 1;
  k.z = a.q, k.zr = s.q_row, k.zg = G;
  k.D1 = s.Dv, k.D2 = s.Dk, k.rev = 1;
  k.s_in = a.dht, k.s1 = 1, k.s2 = s.Dv;
  k.out = G > 1 ? p.pdk : a.dk, k.out_partial = G > 1;
  if (a.dg) k.ex = a.k, k.er = s.k_row, k.eg = G, k.e = p.ek;
  LinChain& v = L.c[2];  // dv, dh0
  v.x = a.k, v.xr = s.k_row, v.xg = G;
  v.y = a.q, v.yr = s.q_row, v.yg = G;
  v.z = a.dout, v.zr = d_row, v.zg = 1;
  v.D1 = s.Dk, v.D2 = s.Dv, v.rev = 1;
  v.s_in = a.dht, v.s_out = a.dh0, v.s1 = s.Dv, v.s2 = 1;
  v.out = a.dv;
  return L;
}

hipError_t launch_lin_bwd_tail(const LinShape& s, const LinBwdArgs& a, const LinBwdParts& p, bool summed, int es,
                               int dots, int64_t segments, int64_t seg, hipStream_t st) {
  if (s.Hv != s.Hk && !summed) {
    ProfScope prof("linear_group_sum", st);
    const int64_t n = s.rows * s.Hk * (s.Dk / 4);
    const dim3 grid(static_cast<unsigned>((n + 255) / 256), 2);
    if (s.out_bf16)
      lin_group_sum_kernel<<<grid, 256, 0, st>>>(p.pdq, p.pdk, static_cast<bf16_t*>(a.dq), static_cast<bf16_t*>(a.dk),
                                                 s.B, s.T, s.rows, s.packed, s.Hk, s.Hv, s.Dk, a.cu);
    else
      lin_group_sum_kernel<<<grid, 256, 0, st>>>(p.pdq, p.pdk, static_cast<float*>(a.dq), static_cast<float*>(a.dk),
                                                 s.B, s.T, s.rows, s.packed, s.Hk, s.Hv, s.Dk, a.cu);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!a.dg) return hipSuccess;
  ProfScope prof("linear_dg", st);
  double* sums = s.head_decay ? p.dgsum : nullptr;
  lin_dg_kernel<<<static_cast<unsigned>(s.B * s.Hv * segments), kDgStep, 0, st>>>(
      p.eq, p.ek, p.xdot, es, dots, a.g, a.dg, sums, s.B, s.T, s.rows, s.packed, s.Hv, segments, seg, a.cu);
  if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (sums) lin_dg_head_kernel<<<s.Hv, 64, 0, st>>>(sums, a.g, a.dg, s.B * segments, s.Hv);
  return hipGetLastError();
}

hipError_t launch_lin_zero(float* p, int n, hipStream_t st) {
  lin_zero_kernel<<<(n + 255) / 256, 256, 0, st>>>(p, n);
  return hipGetLastError();
}

hipError_t launch_lin_token(const LinShape& s, const LinChains& a, hipStream_t st) {
  ProfScope prof("linear_token", st);
  const unsigned grid = static_cast<unsigned>(s.B * s.Hv * lin_slices(s.Dv));
  if (s.io_bf16) lin_token_kernel<bf16_t><<<grid, 256, 0, st>>>(a);
  else lin_token_kernel<float><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_lin_seq(const LinShape& s, const LinChains& a, hipStream_t st) {
  int64_t blocks = 0;
  int rows = 0;
  for (int i = 0; i < a.n; ++i) {
    blocks += a.B * a.Hv * lin_slices(a.c[i].D2);
    rows = a.c[i].D1 > rows ? a.c[i].D1 : rows;
  }
  return s.io_bf16 ? seq_launch<bf16_t>(a, rows, blocks, st) : seq_launch<float>(a, rows, blocks, st);
}

}  // namespace gdr
