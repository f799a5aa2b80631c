// Linear attention with a decay for each head: what its C entry points
// (gdr_linear_api.hip) and kernels (gdr_linear_seq.hip, gdr_linear_chunk.hip)
// share.
//
// Every pass is one kind of chain.  For operands x, y (width D1) and z (width
// D2) and the decay alpha_t = exp(g_t),
//     S_t = alpha_t S_{t-1} + y_t z_t^T  (D1 x D2),   out_t = S_t^T x_t.
//   o  is the chain (q, k, v) forward in time from h0;
//   dq is the chain (dO, v, k) forward in time from h0^T;
//   dv is the chain (k, q, dO) and dk the chain (v, dO, q) backward in time
//      from dht and dht^T, where dS_t = q_t dO_t^T + alpha_{t+1} dS_{t+1};
// dh0 = alpha_1 dS_1 falls out of the dv chain's end, and dg from
//     dg_t = sum_{r >= t} (q_r . dq_r - k_r . dk_r) + <S_T, dS_T>
// (dq, dk per value head), whose row terms e the dq and dk chains leave.
#pragma once

#include <gdr.h>
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdr_internal.h"

namespace gdr {

struct LinShape {
  int64_t B, T;
  int Hk, Hv, Dk, Dv;
  bool io_bf16, out_bf16, head_decay;
  int64_t q_row, k_row, v_row;  // elements between tokens
  // Rows of the VJP's partial results, one for each token: row cu[b] + t for
  // token t of sequence b (`packed`: a dense batch, or a ragged one whose rows
  // are counted), or row b T + t.
  int64_t rows;
  bool packed;
};

struct LinFwdArgs {
  const void *q, *k, *v;
  const float *g, *h0;
  void* o;
  float* ht;
  const int64_t* cu;  // ragged batch row offsets [B + 1], or null
};

struct LinBwdArgs {
  const void *q, *k, *v, *dout;
  const float *g, *h0, *dht;
  void *dq, *dk, *dv;
  float *dg, *dh0;  // either may be null
  const int64_t* cu;
};

// Columns of the state that one workgroup of a chain owns.
constexpr int kLinSlice = 64;
__host__ __device__ inline int lin_slices(int D2) { return (D2 + kLinSlice - 1) / kLinSlice; }

// One chain as its kernels see it.
struct LinChain {
  const void *x, *y, *z;
  int64_t xr, yr, zr;   // elements between tokens
  int xg, yg, zg;       // value heads per head of x, y, z
  int D1, D2, rev;
  const float* s_in;    // [B][Hv] states or null (zeros); element (d1, d2) at d1 * s1 + d2 * s2
  float* s_out;         // null: not wanted
  int s1, s2;
  void* out;            // null: only the state is wanted
  float* sum;           // chunked, over heads: what is added, fp32 [rows][Hv / og][D2]
  int og = 1;           // chunked: value heads to a head of out
  int out_partial;      // 0: out type, rows of the batch; 1: fp32, partial rows (LinShape)
  const void* ex;       // e_t = ex_t . out_t, ex [.., Hv / eg heads, D2], rows er elements apart; null: not wanted
  int64_t er;
  int eg;
  float* e;             // in parts, [slices][Hv][rows] (sequential) or [slices][1 or 2][..] (chunked)
  const float* dot;     // gradient of the last state (element (d1, d2) as for s_in) or null
  float* xdot;          // <last state, dot> in parts, [segments][B][Hv][slices] (sequential) or [..][slices][4]
                        // (chunked); null: not wanted
  // A sequence cut in segments (chunked): the state each segment starts its
  // walk from, [B][Hv][segments][Dk * Dv] (elements as for s_in), which then
  // holds instead of s_in; and the other direction's, which holds instead of dot.
  const float *seg_in, *seg_dot;
  int key;              // chunked: a dq or dk chain of a VJP
};

struct LinChains {
  LinChain c[3];
  int n;                // chains in the launch
  int64_t B, T;
  int64_t rows;         // partial rows (LinShape)
  int packed;
  int Hv, group;        // value heads; those that share a key head
  const float* g;       // null: no decay
  int head_decay;       // g is [Hv]
  int out_bf16;
  const int64_t* cu;
  int64_t segments, seg;  // chunked: segments per sequence and tokens in each
  int sum, head;          // chunked: dq and dk sum over heads, and this launch adds that of each key head
};

#ifdef __HIPCC__
// Chain i of a launch whose kernel takes LinChains as its first argument, read
// from the argument segment by scalar loads.  Indexed as a C++ array, the
// argument would be copied to scratch memory; picked by selects, all three
// chains would fill the scalar registers.
__device__ __forceinline__ LinChain lin_chain(int i) {
  static_assert(offsetof(LinChains, c) == 0 && sizeof(LinChain) % 4 == 0, "chains come first, in whole words");
  typedef const __attribute__((address_space(4))) uint32_t* words;
  const words p = (words)__builtin_amdgcn_kernarg_segment_ptr() + i * (sizeof(LinChain) / 4);
  struct {
    uint32_t w[sizeof(LinChain) / 4];
  } u;
#pragma unroll
  for (unsigned k = 0; k < sizeof(LinChain) / 4; ++k) u.w[k] = p[k];
  return __builtin_bit_cast(LinChain, u);
}
struct LinSpan {
  int64_t t0, len;
};
// Sequence b: its first row and its length, clamped to [0, T].
__device__ __forceinline__ LinSpan lin_span(const int64_t* cu, int64_t b, int64_t T) {
  if (!cu) return LinSpan{b * T, T};
  const int64_t s0 = cu[b], n = cu[b + 1] - s0;
  return LinSpan{s0, n < 0 ? 0 : (n > T ? T : n)};
}
// The partial row of token t of sequence b.
__device__ __forceinline__ int64_t lin_part_row(const LinChains& a, int64_t b, const LinSpan& sp, int64_t t) {
  return (a.packed ? sp.t0 : b * a.T) + t;
}
#endif

LinChains lin_forward_chains(const LinShape& s, const LinFwdArgs& a);

// Carved parts of a backward workspace, common to both algorithms.
struct LinBwdParts {
  float *eq, *ek;    // [slices(Dk)][up to 2][Hv][rows]
  float* xdot;       // [segments][B][Hv][slices(Dk)][4]
  float *pdq, *pdk;  // only where value heads share a key head: [rows][Hv][Dk], or sums [rows][Hk][Dk]
  double* dgsum;     // [B][segments][Hv], only with a decay per head
};
size_t lin_bwd_parts(const LinShape& s, int64_t segments, bool summed, char* base, LinBwdParts* p);  // their bytes
LinChains lin_backward_chains(const LinShape& s, const LinBwdArgs& a, const LinBwdParts& p);

// dq, dk summed over the value heads of a key head; dg from e and xdot.
// `summed`: dq and dk are complete.  Sequences are cut in segments of seg
// tokens, each with its own xdot in `dots` parts; e is in `es` parts.
hipError_t launch_lin_bwd_tail(const LinShape& s, const LinBwdArgs& a, const LinBwdParts& p, bool summed, int es,
                               int dots, int64_t segments, int64_t seg, hipStream_t st);

hipError_t launch_lin_zero(float* p, int n, hipStream_t st);  // p[0 .. n) = 0

hipError_t launch_lin_token(const LinShape& s, const LinChains& a, hipStream_t st);  // forward, T = 1
hipError_t launch_lin_seq(const LinShape& s, const LinChains& a, hipStream_t st);

// Chunked algorithm.  How a problem is cut, and its workspace: the segments'
// states (forward: one direction, backward: both) and factors.
struct LinPlan {
  int64_t segments, seg;
  bool sum;              // backward: dq and dk are summed over a key head's value heads launch by launch
  size_t states, bytes;  // bytes of one direction's segment states; of all
};
LinPlan lin_plan(const LinShape& s, bool backward);
struct LinSegs {
  float *fwd, *rev;    // [B][Hv][segments][Dk * Dv]
  float* factor;       // [B][Hv][segments]
};
LinSegs lin_segs(const LinPlan& p, bool backward, char* base);
hipError_t launch_lin_chunk_fwd(const LinShape& s, const LinPlan& p, const LinFwdArgs& a, char* ws, hipStream_t st);
hipError_t launch_lin_chunk_bwd(const LinShape& s, const LinPlan& p, const LinBwdArgs& a, const LinBwdParts& parts,
                                char* ws, hipStream_t st);

}  // namespace gdr
