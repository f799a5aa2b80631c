// C entry points of the operators beside the gated delta rule (declared in
// include/gdr.h): linear attention with a decay for each head, and the group
// norm of the heads' outputs.  Argument validation, workspace sizes, algorithm
// choice, launches.  Nothing here allocates, frees or synchronises.

#include <gdr.h>

#include "gdr_linear.h"
#include "gdr_norm.h"

namespace {

using gdr::LinShape;

bool misaligned(const void* p, uintptr_t a = 16) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}

bool known(int32_t dtype) { return dtype == GDR_F32 || dtype == GDR_BF16; }

// A row stride: 0 (dense), or at least the row, in whole 16-byte units; 64 rows
// of it lie within 2^30 bytes, which 32-bit offsets reach.
constexpr int64_t kMaxRow = int64_t(1) << 22;
gdr_status check_row(int64_t stride, int64_t dense, int32_t dtype) {
  if (dense > kMaxRow) return GDR_ERR_UNSUPPORTED;
  if (stride == 0) return GDR_OK;
  if (stride < dense) return GDR_ERR_BAD_SHAPE;
  if (stride > kMaxRow) return GDR_ERR_UNSUPPORTED;
  return stride % (dtype == GDR_BF16 ? 8 : 4) ? GDR_ERR_BAD_ALIGNMENT : GDR_OK;
}

// Rows of a VJP's partial results: a ragged batch's own, where the caller
// counts them (kUncounted: it does not) and they are no more than the bound B * T.
constexpr int64_t kUncounted = -1;
bool counted(const gdr_linear_problem* p, int64_t rows) { return rows != kUncounted && rows <= p->B * p->T; }
int64_t partial_rows(const gdr_linear_problem* p, int64_t rows) { return counted(p, rows) ? rows : p->B * p->T; }

gdr_status check(const gdr_linear_problem* p, bool backward, int64_t rows = kUncounted) {
  if (!p) return GDR_ERR_NULL_ARG;
  if (p->B < 0 || p->T < 0 || p->Hk <= 0 || p->Hv <= 0 || p->Dk <= 0 || p->Dv <= 0) return GDR_ERR_BAD_SHAPE;
  if (p->Hv % p->Hk != 0) return GDR_ERR_BAD_SHAPE;
  if (p->Dk % 16 || p->Dv % 16 || p->Dk > 256 || p->Dv > 256) return GDR_ERR_UNSUPPORTED;
  if (!known(p->io_dtype) || !known(p->out_dtype)) return GDR_ERR_UNSUPPORTED;
  if (p->flags & ~static_cast<uint32_t>(GDR_LINEAR_HEAD_DECAY)) return GDR_ERR_UNSUPPORTED;
  if (p->algo < GDR_ALGO_AUTO || p->algo > GDR_ALGO_CHUNKED) return GDR_ERR_UNSUPPORTED;
  const int64_t qk = static_cast<int64_t>(p->Hk) * p->Dk, v = static_cast<int64_t>(p->Hv) * p->Dv;
  for (gdr_status st : {check_row(p->q_row, qk, p->io_dtype), check_row(p->k_row, qk, p->io_dtype),
                        check_row(p->v_row, v, p->io_dtype),
                        check_row(0, static_cast<int64_t>(p->Hv) * p->Dk, p->io_dtype)})
    if (st != GDR_OK) return st;
  // grid limits: a launch has at most 2^32 threads, up to 512 for each slice of
  // the heads' states (segments only where there are few)
  if (p->B > 65535 || p->Hv > 65535 || p->T > 0x7fffffffLL) return GDR_ERR_UNSUPPORTED;
  const int slices = 2 * gdr::lin_slices(p->Dk) + gdr::lin_slices(p->Dv);
  if (p->B * p->Hv * slices > (1 << 22)) return GDR_ERR_UNSUPPORTED;
  // tokens, and in the VJP those of each key head
  if (partial_rows(p, rows) * (backward ? p->Hk : 1) > 0x7fffffffLL) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

LinShape shape_of(const gdr_linear_problem* p, bool ragged = false, int64_t rows = kUncounted) {
  LinShape s;
  s.B = p->B, s.T = p->T, s.Hk = p->Hk, s.Hv = p->Hv, s.Dk = p->Dk, s.Dv = p->Dv;
  s.io_bf16 = p->io_dtype == GDR_BF16;
  s.out_bf16 = p->out_dtype == GDR_BF16;
  s.head_decay = (p->flags & GDR_LINEAR_HEAD_DECAY) != 0;
  s.q_row = p->q_row ? p->q_row : static_cast<int64_t>(p->Hk) * p->Dk;
  s.k_row = p->k_row ? p->k_row : static_cast<int64_t>(p->Hk) * p->Dk;
  s.v_row = p->v_row ? p->v_row : static_cast<int64_t>(p->Hv) * p->Dv;
  s.rows = partial_rows(p, rows);
  s.packed = !ragged || counted(p, rows);
  return s;
}

gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : gdr::record_hip_error(e); }

// Shortest T at which AUTO takes the chunked kernels, which take as long for a
// few tokens as for a chunk.  Token by token against chunked, us, MI355X, 32
// heads of 128 x 128, bf16: forward, 1 sequence 6.9 : 8.8 at T = 2 and 13.8 :
// 8.7 at 8; 8 sequences 12.1 : 18.6 at 4, 17.8 : 18.5 at 8, 28.9 : 18.5 at 16; 64
// sequences 95 : 129 at 4, 125 : 130 at 8, 211 : 136 at 16.  VJP, 8 sequences 45 :
// 72 at 8, 70 : 72 at 16; 64 sequences 325 : 528 at 8, 545 : 531 at 16; 1 sequence
// 22 : 19 at 8.  fp32, 8 sequences of 8 heads: forward 7.6 : 11.1 at 4, 11.2 : 11.1
// at 8; VJP 19.7 : 27.4 at 8, 27.7 : 27.6 at 16.
constexpr int64_t kAutoForwardT = 8, kAutoBackwardT = 16;
bool chunked(const gdr_linear_problem* p, bool backward) {
  if (p->algo != GDR_ALGO_AUTO) return p->algo == GDR_ALGO_CHUNKED;
  return p->T >= (backward ? kAutoBackwardT : kAutoForwardT);
}

// Workspace of a call: the parts of a backward, then the chunked algorithm's
// segment states.
size_t forward_bytes(const gdr_linear_problem* p) {
  return chunked(p, false) ? gdr::lin_plan(shape_of(p), false).bytes : 0;
}
size_t backward_bytes(const gdr_linear_problem* p, int64_t rows) {
  const LinShape s = shape_of(p, rows != kUncounted, rows);
  const gdr::LinPlan plan = gdr::lin_plan(s, true);
  const bool chunk = chunked(p, true);
  gdr::LinBwdParts parts;
  const size_t used = gdr::lin_bwd_parts(s, chunk ? plan.segments : 1, chunk && plan.sum, nullptr, &parts);
  return used + (chunk ? plan.bytes : 0);
}

gdr_status check_ws(const void* ws, size_t have, size_t need) {
  if (misaligned(ws, 256)) return GDR_ERR_BAD_ALIGNMENT;
  if (need == 0) return GDR_OK;
  if (!ws) return GDR_ERR_NULL_ARG;
  return have < need ? GDR_ERR_WORKSPACE_TOO_SMALL : GDR_OK;
}

gdr_status linear_forward(const gdr_linear_problem* p, const int64_t* cu, bool ragged, const void* q, const void* k,
                          const void* v, const float* g, const float* h0, void* o, float* ht, void* ws,
                          size_t ws_bytes, void* hip_stream) {
  gdr_status st = check(p, false);
  if (st != GDR_OK) return st;
  const LinShape s = shape_of(p);
  const bool empty = s.B == 0 || s.T == 0;
  if (!empty && (!q || !k || !v || !o)) return GDR_ERR_NULL_ARG;
  if (ragged && !empty && !cu) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {q, k, v, static_cast<const void*>(h0), static_cast<const void*>(o),
                          static_cast<const void*>(ht)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(g, 4) || misaligned(cu, 8)) return GDR_ERR_BAD_ALIGNMENT;
  if ((st = check_ws(ws, ws_bytes, empty ? 0 : forward_bytes(p))) != GDR_OK) return st;
  if (s.B == 0 || (s.T == 0 && (!ht || ht == h0))) return GDR_OK;
  const gdr::LinFwdArgs a{q, k, v, g, h0, o, ht, cu};
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (s.T > 0 && chunked(p, false))
    return done(gdr::launch_lin_chunk_fwd(s, gdr::lin_plan(s, false), a, static_cast<char*>(ws), stream));
  const gdr::LinChains chains = gdr::lin_forward_chains(s, a);
  // the sequential algorithm adds in one order however a sequence is cut into calls
  const bool token = s.T == 1 && p->algo == GDR_ALGO_AUTO;
  return done(token ? gdr::launch_lin_token(s, chains, stream) : gdr::launch_lin_seq(s, chains, stream));
}

bool nothing(const gdr_linear_problem* p, int64_t rows) { return p->B == 0 || p->T == 0 || rows == 0; }

gdr_status linear_backward(const gdr_linear_problem* p, const int64_t* cu, bool ragged, int64_t rows, const void* q,
                           const void* k, const void* v, const float* g, const float* h0, const void* dout,
                           const float* dht, void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws,
                           size_t ws_bytes, void* hip_stream) {
  gdr_status st = check(p, true, rows);
  if (st != GDR_OK) return st;
  const LinShape s = shape_of(p, ragged, rows);
  const bool empty = nothing(p, rows);
  if (!empty && (!q || !k || !v || !dout || !dq || !dk || !dv)) return GDR_ERR_NULL_ARG;
  if (ragged && !empty && !cu) return GDR_ERR_NULL_ARG;
  if (dg && !g) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {q, k, v, static_cast<const void*>(h0), dout, static_cast<const void*>(dht),
                          static_cast<const void*>(dq), static_cast<const void*>(dk), static_cast<const void*>(dv),
                          static_cast<const void*>(dh0)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(g, 4) || misaligned(dg, 4) || misaligned(cu, 8)) return GDR_ERR_BAD_ALIGNMENT;
  if ((st = check_ws(ws, ws_bytes, empty ? 0 : backward_bytes(p, rows))) != GDR_OK) return st;
  const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  const gdr::LinBwdArgs a{q, k, v, dout, g, h0, dht, dq, dk, dv, dg, dh0, cu};
  const bool chunk = !empty && chunked(p, true);
  const gdr::LinPlan plan = chunk ? gdr::lin_plan(s, true) : gdr::LinPlan{1, s.T, false, 0, 0};
  gdr::LinBwdParts parts;
  const size_t used = gdr::lin_bwd_parts(s, plan.segments, plan.sum, static_cast<char*>(ws), &parts);
  if (chunk)
    return done(gdr::launch_lin_chunk_bwd(s, plan, a, parts, static_cast<char*>(ws) + used, stream));
  if (empty) {
    if (s.B > 0 && dh0) {  // the state passes through
      gdr::LinChains all = gdr::lin_backward_chains(s, a, parts), one = all;
      one.c[0] = all.c[2], one.n = 1, one.T = 0;
      if (hipError_t e = gdr::launch_lin_seq(s, one, stream); e != hipSuccess) return done(e);
    }
    return dg && s.head_decay ? done(gdr::launch_lin_zero(dg, s.Hv, stream)) : GDR_OK;
  }
  if (hipError_t e = gdr::launch_lin_seq(s, gdr::lin_backward_chains(s, a, parts), stream); e != hipSuccess)
    return done(e);
  const int parted = gdr::lin_slices(s.Dk);
  return done(gdr::launch_lin_bwd_tail(s, a, parts, false, parted, parted, 1, s.T, stream));
}

gdr_status check(const gdr_norm_problem* p) {
  if (!p) return GDR_ERR_NULL_ARG;
  if (p->rows < 0 || p->groups <= 0 || p->channels <= 0) return GDR_ERR_BAD_SHAPE;
  if (p->channels % 8 || p->channels > 512) return GDR_ERR_UNSUPPORTED;
  if (!known(p->io_dtype) || !known(p->out_dtype)) return GDR_ERR_UNSUPPORTED;
  if (p->flags & ~static_cast<uint32_t>(GDR_NORM_CENTER | GDR_NORM_SILU | GDR_NORM_SHARED_WEIGHT))
    return GDR_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.f)) return GDR_ERR_BAD_SHAPE;
  if (p->groups > 65535 || p->rows > (int64_t(1) << 40)) return GDR_ERR_UNSUPPORTED;
  const int64_t row = static_cast<int64_t>(p->groups) * p->channels;
  gdr_status st = check_row(p->x_row, row, p->io_dtype);
  return st != GDR_OK ? st : check_row(p->z_row, row, p->io_dtype);
}

gdr::NormArgs norm_args(const gdr_norm_problem* p) {
  gdr::NormArgs a{};
  const int64_t row = static_cast<int64_t>(p->groups) * p->channels;
  a.rows = p->rows, a.G = p->groups, a.D = p->channels, a.eps = p->eps;
  a.x_row = p->x_row ? p->x_row : row;
  a.z_row = p->z_row ? p->z_row : row;
  a.io_bf16 = p->io_dtype == GDR_BF16, a.out_bf16 = p->out_dtype == GDR_BF16;
  a.center = p->flags & GDR_NORM_CENTER, a.silu = p->flags & GDR_NORM_SILU;
  a.shared = p->flags & GDR_NORM_SHARED_WEIGHT;
  return a;
}

}  // namespace

extern "C" {

gdr_status gdr_linear_forward_workspace(const gdr_linear_problem* p, size_t* bytes) {
  const gdr_status st = check(p, false);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_NULL_ARG;
  *bytes = p->B == 0 || p->T == 0 ? 0 : forward_bytes(p);
  return GDR_OK;
}

gdr_status gdr_linear_backward_workspace(const gdr_linear_problem* p, size_t* bytes) {
  const gdr_status st = check(p, true);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_NULL_ARG;
  *bytes = nothing(p, kUncounted) ? 0 : backward_bytes(p, kUncounted);
  return GDR_OK;
}

gdr_status gdr_linear_backward_varlen_workspace(const gdr_linear_problem* p, int64_t rows, size_t* bytes) {
  if (rows < 0) return p ? GDR_ERR_BAD_SHAPE : GDR_ERR_NULL_ARG;
  const gdr_status st = check(p, true, rows);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_NULL_ARG;
  *bytes = nothing(p, rows) ? 0 : backward_bytes(p, rows);
  return GDR_OK;
}

gdr_status gdr_linear_forward(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                              const float* g, const float* h0, void* o, float* ht, void* ws, size_t ws_bytes,
                              void* hip_stream) {
  return linear_forward(p, nullptr, false, q, k, v, g, h0, o, ht, ws, ws_bytes, hip_stream);
}

gdr_status gdr_linear_forward_varlen(const gdr_linear_problem* p, const int64_t* cu_seqlens, const void* q,
                                     const void* k, const void* v, const float* g, const float* h0, void* o,
                                     float* ht, void* ws, size_t ws_bytes, void* hip_stream) {
  return linear_forward(p, cu_seqlens, true, q, k, v, g, h0, o, ht, ws, ws_bytes, hip_stream);
}

gdr_status gdr_linear_backward(const gdr_linear_problem* p, const void* q, const void* k, const void* v,
                               const float* g, const float* h0, const void* dout, const float* dht, void* dq,
                               void* dk, void* dv, float* dg, float* dh0, void* ws, size_t ws_bytes,
                               void* hip_stream) {
  return linear_backward(p, nullptr, false, kUncounted, q, k, v, g, h0, dout, dht, dq, dk, dv, dg, dh0, ws,
                         ws_bytes, hip_stream);
}

gdr_status gdr_linear_backward_varlen(const gdr_linear_problem* p, const int64_t* cu_seqlens, const void* q,
                                      const void* k, const void* v, const float* g, const float* h0,
                                      const void* dout, const float* dht, void* dq, void* dk, void* dv, float* dg,
                                      float* dh0, void* ws, size_t ws_bytes, void* hip_stream) {
  return linear_backward(p, cu_seqlens, true, kUncounted, q, k, v, g, h0, dout, dht, dq, dk, dv, dg, dh0, ws,
                         ws_bytes, hip_stream);
}

gdr_status gdr_linear_backward_varlen_rows(const gdr_linear_problem* p, int64_t rows, const int64_t* cu_seqlens,
                                           const void* q, const void* k, const void* v, const float* g,
                                           const float* h0, const void* dout, const float* dht, void* dq, void* dk,
                                           void* dv, float* dg, float* dh0, void* ws, size_t ws_bytes,
                                           void* hip_stream) {
  if (rows < 0) return p ? GDR_ERR_BAD_SHAPE : GDR_ERR_NULL_ARG;
  return linear_backward(p, cu_seqlens, true, rows, q, k, v, g, h0, dout, dht, dq, dk, dv, dg, dh0, ws, ws_bytes,
                         hip_stream);
}

gdr_status gdr_group_norm_forward(const gdr_norm_problem* p, const void* x, const float* weight, const float* bias,
                                  const void* z, void* y, void* hip_stream) {
  const gdr_status st = check(p);
  if (st != GDR_OK) return st;
  if (z && (p->flags & GDR_NORM_SILU)) return GDR_ERR_UNSUPPORTED;
  if (p->rows > 0 && (!x || !y)) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {x, z, static_cast<const void*>(y), static_cast<const void*>(weight),
                          static_cast<const void*>(bias)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (p->rows == 0) return GDR_OK;
  gdr::NormArgs a = norm_args(p);
  a.x = x, a.w = weight, a.b = bias, a.z = z, a.y = y;
  return done(gdr::launch_norm_fwd(a, static_cast<hipStream_t>(hip_stream)));
}

gdr_status gdr_group_norm_backward_workspace(const gdr_norm_problem* p, size_t* bytes) {
  const gdr_status st = check(p);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_NULL_ARG;
  *bytes = gdr::norm_bwd_workspace(norm_args(p));
  return GDR_OK;
}

gdr_status gdr_group_norm_backward(const gdr_norm_problem* p, const void* x, const float* weight, const float* bias,
                                   const void* z, const void* dy, void* dx, void* dz, float* dweight, float* dbias,
                                   void* ws, size_t ws_bytes, void* hip_stream) {
  gdr_status st = check(p);
  if (st != GDR_OK) return st;
  if (z && (p->flags & GDR_NORM_SILU)) return GDR_ERR_UNSUPPORTED;
  if (p->rows > 0 && (!x || !dy || !dx || (z && !dz))) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {x, z, dy, static_cast<const void*>(dx), static_cast<const void*>(dz),
                          static_cast<const void*>(weight), static_cast<const void*>(bias),
                          static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (p->rows == 0 && !dweight && !dbias) return GDR_OK;
  gdr::NormArgs a = norm_args(p);
  if ((st = check_ws(ws, ws_bytes, dweight || dbias ? gdr::norm_bwd_workspace(a) : 0)) != GDR_OK) return st;
  a.x = x, a.w = weight, a.b = bias, a.z = z, a.dy = dy;
  a.dx = dx, a.dz = dz, a.dw = dweight, a.db = dbias, a.part = static_cast<float*>(ws);
  return done(gdr::launch_norm_bwd(a, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
