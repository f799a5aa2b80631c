// C entry points of the attention layer's operators (declared in include/gdr.h):
// rotary positions, the paged cache's append and single-token attention, and
// attention over whole sequences.  Argument validation, workspace sizes,
// launches.  Nothing here allocates, frees or synchronises.

#include <gdr.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "gdr_attn.h"

namespace {

bool misaligned(const void* p, uintptr_t a = 16) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) != 0;
}
bool known(int32_t dtype) { return dtype == GDR_F32 || dtype == GDR_BF16; }
int per16(int32_t dtype) { return dtype == GDR_BF16 ? 8 : 4; }
gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : gdr::record_hip_error(e); }

constexpr int64_t kMaxRows = 0x7fffffffLL;
constexpr int64_t kMaxT = (int64_t(1) << 22) - 128;  // tokens of a sequence
constexpr int64_t kMaxLen = int64_t(1) << 30;  // tokens of a sequence in a cache

// A row distance: 0 (dense), or at least the row, in whole 16-byte units.  Where tiles
// of rows are loaded, the 128 rows of one lie within 2^31 bytes, which 32-bit offsets
// reach; where rows are addressed one by one (in 64 bits) they may lie further apart,
// as one token of each of a batch's long sequences does.
constexpr int64_t kMaxRow = int64_t(1) << 22, kFarRow = int64_t(1) << 40;
gdr_status check_row(int64_t stride, int64_t dense, int32_t dtype, int64_t most = kFarRow) {
  if (dense > kMaxRow) return GDR_ERR_UNSUPPORTED;
  if (stride == 0) return GDR_OK;
  if (stride < dense) return GDR_ERR_BAD_SHAPE;
  if (stride > most) return GDR_ERR_UNSUPPORTED;
  return stride % per16(dtype) ? GDR_ERR_BAD_ALIGNMENT : GDR_OK;
}
gdr_status first_of(std::initializer_list<gdr_status> all) {
  for (gdr_status st : all)
    if (st != GDR_OK) return st;
  return GDR_OK;
}
int64_t row_of(int64_t stride, int64_t heads, int64_t D) { return stride ? stride : heads * D; }

gdr_status check_dim(int32_t D) {
  if (D <= 0) return GDR_ERR_BAD_SHAPE;
  return D % 16 || D > 256 ? GDR_ERR_UNSUPPORTED : GDR_OK;
}

gdr_status check(const gdr_rotary& r, int32_t D) {
  if (r.R < 0 || r.R > D || r.axes < 1) return GDR_ERR_BAD_SHAPE;
  if (r.R % 16 || r.axes > 4) return GDR_ERR_UNSUPPORTED;
  if (r.flags & ~static_cast<uint32_t>(GDR_ROTARY_ADJACENT | GDR_ROTARY_CYCLED)) return GDR_ERR_UNSUPPORTED;
  if (r.axes == 1) return GDR_OK;
  int64_t sum = 0;
  for (int i = 0; i < r.axes; ++i) {
    const int64_t n = r.section[i];
    if (n < 0) return GDR_ERR_BAD_SHAPE;
    // the last of an axis' pairs, taken in turns, is one of the R / 2
    if ((r.flags & GDR_ROTARY_CYCLED) && i > 0 && n > 0 && r.axes * (n - 1) + i >= r.R / 2) return GDR_ERR_BAD_SHAPE;
    sum += n;
  }
  return sum == r.R / 2 ? GDR_OK : GDR_ERR_BAD_SHAPE;
}

gdr_status check(const gdr_cache& c) {
  if (c.pages < 0 || c.page_size <= 0 || c.Hk <= 0 || c.max_pages < 0 || c.table_row < 0) return GDR_ERR_BAD_SHAPE;
  if (gdr_status st = check_dim(c.D); st != GDR_OK) return st;
  if (!known(c.dtype) || c.pages > 0x7fffffffLL || c.Hk > 65535) return GDR_ERR_UNSUPPORTED;
  if (c.table_row != 0 && c.table_row < c.max_pages) return GDR_ERR_BAD_SHAPE;
  struct Dim {
    int64_t stride, n;
  } dims[3] = {{c.page_stride, c.pages}, {c.token_stride, c.page_size}, {c.head_stride, c.Hk}};
  if (c.page_stride == 0 && c.token_stride == 0 && c.head_stride == 0) {
    dims[2].stride = c.D;
    dims[1].stride = static_cast<int64_t>(c.Hk) * c.D;
    if (c.page_size > (int64_t(1) << 40) / dims[1].stride) return GDR_ERR_UNSUPPORTED;
    dims[0].stride = c.page_size * dims[1].stride;
  }
  // no two elements in one place: each step clears what the smaller steps span
  std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
  __int128 spans = c.D;
  for (const Dim& d : dims) {
    if (d.n <= 1) continue;
    if (d.stride < spans) return GDR_ERR_BAD_SHAPE;
    if (d.stride % per16(c.dtype)) return GDR_ERR_BAD_ALIGNMENT;
    spans += static_cast<__int128>(d.stride) * (d.n - 1);
  }
  return spans * (16 / per16(c.dtype)) > (static_cast<__int128>(64) << 30) ? GDR_ERR_UNSUPPORTED : GDR_OK;
}

gdr::CacheView view_of(const gdr_cache& c, const int32_t* table, const int64_t* lengths) {
  gdr::CacheView v{};
  v.pages = c.pages, v.page_size = c.page_size, v.Hk = c.Hk, v.D = c.D, v.max_pages = c.max_pages;
  v.page_stride = c.page_stride, v.token_stride = c.token_stride, v.head_stride = c.head_stride;
  if (c.page_stride == 0 && c.token_stride == 0 && c.head_stride == 0) {
    v.head_stride = c.D;
    v.token_stride = static_cast<int64_t>(c.Hk) * c.D;
    v.page_stride = c.page_size * v.token_stride;
  }
  v.table_row = c.table_row ? c.table_row : c.max_pages;
  v.table = table, v.lengths = lengths;
  return v;
}

void set_rotary(gdr::RotArgs& a, const gdr_rotary& r) {
  a.R = r.R, a.axes = r.axes;
  for (int i = 0; i < 4; ++i) a.section[i] = r.section[i];
  a.adjacent = r.flags & GDR_ROTARY_ADJACENT, a.cycled = r.flags & GDR_ROTARY_CYCLED;
}

gdr_status rotary(const gdr_rotary_problem* p, const void* q, const void* k, const int64_t* pos, const float* freq,
                  void* qo, void* ko, bool back, void* hip_stream) {
  if (!p) return GDR_ERR_NULL_ARG;
  if (p->rows < 0 || p->Hq <= 0 || p->Hk < 0) return GDR_ERR_BAD_SHAPE;
  gdr_status st = first_of({check_dim(p->D), check(p->rot, p->D)});
  if (st != GDR_OK) return st;
  if (!known(p->io_dtype) || !known(p->out_dtype) || p->rows > kMaxRows) return GDR_ERR_UNSUPPORTED;
  const int64_t nq = static_cast<int64_t>(p->Hq) * p->D, nk = static_cast<int64_t>(p->Hk) * p->D;
  st = first_of({check_row(p->q_row, nq, p->io_dtype), check_row(p->qo_row, nq, p->out_dtype),
                 check_row(p->Hk ? p->k_row : 0, nk, p->io_dtype), check_row(p->Hk ? p->ko_row : 0, nk, p->out_dtype)});
  if (st != GDR_OK) return st;
  if (p->rows > 0 && (!q || !qo || (p->Hk && (!k || !ko)) || (p->rot.R && (!pos || !freq)))) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {q, k, static_cast<const void*>(qo), static_cast<const void*>(ko)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(pos, 8) || misaligned(freq, 4)) return GDR_ERR_BAD_ALIGNMENT;
  if (p->rows == 0) return GDR_OK;
  gdr::RotArgs a{};
  set_rotary(a, p->rot);
  a.q = q, a.k = k, a.pos = pos, a.freq = freq, a.qo = qo, a.ko = ko, a.rows = p->rows;
  a.Hq = p->Hq, a.Hk = p->Hk, a.D = p->D, a.back = back;
  a.q_row = row_of(p->q_row, p->Hq, p->D), a.k_row = row_of(p->k_row, p->Hk, p->D);
  a.qo_row = row_of(p->qo_row, p->Hq, p->D), a.ko_row = row_of(p->ko_row, p->Hk, p->D);
  a.io_bf16 = p->io_dtype == GDR_BF16, a.out_bf16 = p->out_dtype == GDR_BF16;
  return done(gdr::launch_rotary(a, static_cast<hipStream_t>(hip_stream)));
}

gdr_status append(const gdr_append_problem* p, const int64_t* cu, bool ragged, const int64_t* lengths,
                  const int32_t* table, const void* q, const void* k, const void* v, const int64_t* pos,
                  const float* freq, void* qo, void* kc, void* vc, void* hip_stream) {
  if (!p) return GDR_ERR_NULL_ARG;
  if (p->B < 0 || p->T < 0 || p->Hq < 0 || (ragged && p->rows < 0)) return GDR_ERR_BAD_SHAPE;
  const gdr_cache& c = p->cache;
  gdr_status st = first_of({check(c), check(p->rot, c.D)});
  if (st != GDR_OK) return st;
  if (!known(p->io_dtype) || p->B > 65535) return GDR_ERR_UNSUPPORTED;
  if (p->T > kMaxRows || (ragged ? p->rows : p->B * p->T) > kMaxRows) return GDR_ERR_UNSUPPORTED;
  const int64_t nq = static_cast<int64_t>(p->Hq) * c.D, nk = static_cast<int64_t>(c.Hk) * c.D;
  st = first_of({check_row(p->Hq ? p->q_row : 0, nq, p->io_dtype), check_row(p->k_row, nk, p->io_dtype),
                 check_row(p->v_row, nk, p->io_dtype)});
  if (st != GDR_OK) return st;
  const int64_t rows = ragged ? p->rows : p->B * p->T;
  const bool empty = rows == 0 || p->B == 0 || p->T == 0;
  // a cache without pages has no buffers: nothing is stored, q is turned all the same
  if (!empty && (!k || !v || (c.pages && (!kc || !vc)) || !lengths || (!table && c.max_pages) ||
                 (p->Hq && (!q || !qo)) || (ragged && !cu) || (p->rot.R && !freq)))
    return GDR_ERR_NULL_ARG;
  if (p->rot.R && p->rot.axes > 1 && !pos && !empty) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {q, k, v, static_cast<const void*>(qo), static_cast<const void*>(kc),
                          static_cast<const void*>(vc)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(pos, 8) || misaligned(lengths, 8) || misaligned(cu, 8) || misaligned(table, 4) || misaligned(freq, 4))
    return GDR_ERR_BAD_ALIGNMENT;
  if (empty) return GDR_OK;
  gdr::RotArgs a{};
  set_rotary(a, p->rot);
  a.q = q, a.k = k, a.v = v, a.pos = pos, a.cu = ragged ? cu : nullptr, a.freq = freq;
  a.qo = qo, a.ko = kc, a.vc = vc, a.cache = view_of(c, table, lengths);
  a.rows = rows, a.B = p->B, a.T = p->T, a.Hq = p->Hq, a.Hk = c.Hk, a.D = c.D;
  a.q_row = row_of(p->q_row, p->Hq, c.D), a.qo_row = nq;
  a.k_row = row_of(p->k_row, c.Hk, c.D), a.v_row = row_of(p->v_row, c.Hk, c.D);
  a.append = true, a.io_bf16 = p->io_dtype == GDR_BF16, a.out_bf16 = c.dtype == GDR_BF16;
  return done(gdr::launch_rotary(a, static_cast<hipStream_t>(hip_stream)));
}

gdr_status check(const gdr_cache_attention_problem* p) {
  if (!p) return GDR_ERR_NULL_ARG;
  const gdr_cache& c = p->cache;
  if (p->B < 0 || p->Hq <= 0 || p->max_len < 0 || p->window < 0 || p->sinks < 0) return GDR_ERR_BAD_SHAPE;
  if (gdr_status st = check(c); st != GDR_OK) return st;
  if (p->Hq % c.Hk || !(p->scale > 0.f) || std::isinf(p->scale)) return GDR_ERR_BAD_SHAPE;
  if (p->max_len > static_cast<int64_t>(c.max_pages) * c.page_size) return GDR_ERR_BAD_SHAPE;
  if (!known(p->out_dtype) || p->B > 65535 || p->Hq > 65535 || p->B * p->Hq > (1 << 22)) return GDR_ERR_UNSUPPORTED;
  if (p->max_len > kMaxLen || (!p->max_len && static_cast<int64_t>(c.max_pages) * c.page_size > kMaxLen))
    return GDR_ERR_UNSUPPORTED;
  return check_row(p->q_row, static_cast<int64_t>(p->Hq) * c.D, c.dtype);
}
gdr::CacheAttnArgs args_of(const gdr_cache_attention_problem* p, const int32_t* table, const int64_t* lengths) {
  gdr::CacheAttnArgs a{};
  a.cache = view_of(p->cache, table, lengths);
  a.B = p->B, a.Hq = p->Hq, a.q_row = row_of(p->q_row, p->Hq, p->cache.D), a.scale = p->scale;
  a.max_len = p->max_len ? p->max_len : static_cast<int64_t>(p->cache.max_pages) * p->cache.page_size;
  // bounds past every length change nothing
  a.sinks = std::min(p->sinks, a.max_len);
  a.window = p->window >= a.max_len ? 0 : p->window;
  a.bf16 = p->cache.dtype == GDR_BF16, a.out_bf16 = p->out_dtype == GDR_BF16;
  return a;
}

gdr_status check_ws(const void* ws, size_t have, size_t need) {
  if (misaligned(ws, 256)) return GDR_ERR_BAD_ALIGNMENT;
  if (need == 0) return GDR_OK;
  if (!ws) return GDR_ERR_NULL_ARG;
  return have < need ? GDR_ERR_WORKSPACE_TOO_SMALL : GDR_OK;
}

gdr_status check(const gdr_attention_problem* p, int64_t rows) {
  if (!p) return GDR_ERR_NULL_ARG;
  if (p->B < 0 || p->T < 0 || rows < 0 || p->Hq <= 0 || p->Hk <= 0 || p->window < 0 || p->sinks < 0)
    return GDR_ERR_BAD_SHAPE;
  if (p->Hq % p->Hk || !(p->scale > 0.f) || std::isinf(p->scale)) return GDR_ERR_BAD_SHAPE;
  if (gdr_status st = check_dim(p->D); st != GDR_OK) return st;
  if (!known(p->io_dtype) || !known(p->out_dtype)) return GDR_ERR_UNSUPPORTED;
  // a grid has less than 2^16 blocks (of 64 rows or more) and 2^32 threads
  if (p->B > 65535 || p->Hq > 65535 || p->T > kMaxT || rows > kMaxRows) return GDR_ERR_UNSUPPORTED;
  if (p->B * p->Hq * ((p->T + 127) / 128) > (1 << 22)) return GDR_ERR_UNSUPPORTED;
  const int64_t q = static_cast<int64_t>(p->Hq) * p->D, k = static_cast<int64_t>(p->Hk) * p->D;
  return first_of({check_row(p->q_row, q, p->io_dtype, kMaxRow), check_row(p->k_row, k, p->io_dtype, kMaxRow),
                   check_row(p->v_row, k, p->io_dtype, kMaxRow)});
}
// B * T, where it is no larger than it may be
int64_t dense_rows(const gdr_attention_problem* p) {
  if (!p || p->B < 0 || p->T < 0) return 0;
  return p->B > 65535 || p->T > kMaxT ? kMaxRows + 1 : p->B * p->T;
}
gdr::AttnArgs args_of(const gdr_attention_problem* p, int64_t rows) {
  gdr::AttnArgs a{};
  a.B = p->B, a.T = p->T, a.rows = rows, a.Hq = p->Hq, a.Hk = p->Hk, a.D = p->D, a.scale = p->scale;
  a.q_row = row_of(p->q_row, p->Hq, p->D);
  a.k_row = row_of(p->k_row, p->Hk, p->D), a.v_row = row_of(p->v_row, p->Hk, p->D);
  // bounds past every length change nothing
  a.sinks = std::min(p->sinks, p->T);
  a.window = p->window >= p->T ? 0 : p->window;
  a.io_bf16 = p->io_dtype == GDR_BF16, a.out_bf16 = p->out_dtype == GDR_BF16;
  return a;
}

gdr_status attention_forward(const gdr_attention_problem* p, const int64_t* cu, bool ragged, const void* q,
                             const void* k, const void* v, void* o, float* lse, void* hip_stream) {
  const int64_t rows = ragged ? 0 : dense_rows(p);
  const gdr_status st = check(p, rows);
  if (st != GDR_OK) return st;
  const bool empty = p->B == 0 || p->T == 0;
  if (!empty && (!q || !k || !v || !o || !lse || (ragged && !cu))) return GDR_ERR_NULL_ARG;
  for (const void* ptr : {q, k, v, static_cast<const void*>(o)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(lse, 4) || misaligned(cu, 8)) return GDR_ERR_BAD_ALIGNMENT;
  if (empty) return GDR_OK;
  gdr::AttnArgs a = args_of(p, rows);
  a.q = q, a.k = k, a.v = v, a.o = o, a.lse = lse, a.cu = ragged ? cu : nullptr;
  return done(gdr::launch_attn_fwd(a, static_cast<hipStream_t>(hip_stream)));
}

gdr_status attention_backward(const gdr_attention_problem* p, int64_t rows, const int64_t* cu, bool ragged,
                              const void* q, const void* k, const void* v, const void* o, const float* lse,
                              const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                              void* hip_stream) {
  gdr_status st = check(p, rows);
  if (st != GDR_OK) return st;
  const bool empty = p->B == 0 || p->T == 0 || rows == 0;
  if (!empty && (!q || !k || !v || !o || !lse || !dout || !dq || !dk || !dv || (ragged && !cu)))
    return GDR_ERR_NULL_ARG;
  for (const void* ptr : {q, k, v, o, dout, static_cast<const void*>(dq), static_cast<const void*>(dk),
                          static_cast<const void*>(dv)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(lse, 4) || misaligned(cu, 8)) return GDR_ERR_BAD_ALIGNMENT;
  gdr::AttnArgs a = args_of(p, rows);
  if ((st = check_ws(ws, ws_bytes, empty ? 0 : gdr::attn_bwd_workspace(a))) != GDR_OK) return st;
  if (empty) return GDR_OK;
  a.q = q, a.k = k, a.v = v, a.out = o, a.lse_in = lse, a.dout = dout, a.cu = ragged ? cu : nullptr;
  a.dq = dq, a.dk = dk, a.dv = dv, a.ws = static_cast<char*>(ws);
  return done(gdr::launch_attn_bwd(a, static_cast<hipStream_t>(hip_stream)));
}

}  // namespace

extern "C" {

gdr_status gdr_rotary_forward(const gdr_rotary_problem* p, const void* q, const void* k, const int64_t* pos,
                              const float* freq, void* q_out, void* k_out, void* hip_stream) {
  return rotary(p, q, k, pos, freq, q_out, k_out, false, hip_stream);
}

gdr_status gdr_rotary_backward(const gdr_rotary_problem* p, const void* dq_out, const void* dk_out,
                               const int64_t* pos, const float* freq, void* dq, void* dk, void* hip_stream) {
  return rotary(p, dq_out, dk_out, pos, freq, dq, dk, true, hip_stream);
}

gdr_status gdr_cache_append(const gdr_append_problem* p, const int64_t* lengths, const int32_t* table, const void* q,
                            const void* k, const void* v, const int64_t* pos, const float* freq, void* q_out,
                            void* k_cache, void* v_cache, void* hip_stream) {
  return append(p, nullptr, false, lengths, table, q, k, v, pos, freq, q_out, k_cache, v_cache, hip_stream);
}

gdr_status gdr_cache_append_varlen(const gdr_append_problem* p, const int64_t* cu_seqlens, const int64_t* lengths,
                                   const int32_t* table, const void* q, const void* k, const void* v,
                                   const int64_t* pos, const float* freq, void* q_out, void* k_cache, void* v_cache,
                                   void* hip_stream) {
  return append(p, cu_seqlens, true, lengths, table, q, k, v, pos, freq, q_out, k_cache, v_cache, hip_stream);
}

gdr_status gdr_cache_attention_workspace(const gdr_cache_attention_problem* p, size_t* bytes) {
  const gdr_status st = check(p);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_NULL_ARG;
  *bytes = p->B == 0 ? 0 : gdr::cache_attn_workspace(args_of(p, nullptr, nullptr));
  return GDR_OK;
}

gdr_status gdr_cache_attention(const gdr_cache_attention_problem* p, const void* q, const void* k_cache,
                               const void* v_cache, const int32_t* table, const int64_t* lengths, void* o, float* lse,
                               void* ws, size_t ws_bytes, void* hip_stream) {
  gdr_status st = check(p);
  if (st != GDR_OK) return st;
  if (p->B > 0) {
    if (!q || !o || !lengths) return GDR_ERR_NULL_ARG;
    if (p->cache.max_pages > 0 && !table) return GDR_ERR_NULL_ARG;
    if (p->cache.max_pages > 0 && p->cache.pages > 0 && (!k_cache || !v_cache)) return GDR_ERR_NULL_ARG;
  }
  for (const void* ptr : {q, k_cache, v_cache, static_cast<const void*>(o)})
    if (misaligned(ptr)) return GDR_ERR_BAD_ALIGNMENT;
  if (misaligned(table, 4) || misaligned(lengths, 8) || misaligned(lse, 4)) return GDR_ERR_BAD_ALIGNMENT;
  gdr::CacheAttnArgs a = args_of(p, table, lengths);
  if ((st = check_ws(ws, ws_bytes, p->B == 0 ? 0 : gdr::cache_attn_workspace(a))) != GDR_OK) return st;
  if (p->B == 0) return GDR_OK;
  a.q = q, a.kc = k_cache, a.vc = v_cache, a.o = o, a.lse = lse, a.part = static_cast<float*>(ws);
  return done(gdr::launch_cache_attn(a, static_cast<hipStream_t>(hip_stream)));
}

gdr_status gdr_attention_forward(const gdr_attention_problem* p, const void* q, const void* k, const void* v, void* o,
                                 float* lse, void* hip_stream) {
  return attention_forward(p, nullptr, false, q, k, v, o, lse, hip_stream);
}

gdr_status gdr_attention_forward_varlen(const gdr_attention_problem* p, const int64_t* cu_seqlens, const void* q,
                                        const void* k, const void* v, void* o, float* lse, void* hip_stream) {
  return attention_forward(p, cu_seqlens, true, q, k, v, o, lse, hip_stream);
}

gdr_status gdr_attention_backward_workspace(const gdr_attention_problem* p, int64_t rows, size_t* bytes) {
  const gdr_status st = check(p, rows);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_NULL_ARG;
  *bytes = p->B == 0 || p->T == 0 || rows == 0 ? 0 : gdr::attn_bwd_workspace(args_of(p, rows));
  return GDR_OK;
}

gdr_status gdr_attention_backward(const gdr_attention_problem* p, const void* q, const void* k, const void* v,
                                  const void* o, const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                  void* ws, size_t ws_bytes, void* hip_stream) {
  return attention_backward(p, dense_rows(p), nullptr, false, q, k, v, o, lse, dout, dq, dk, dv, ws, ws_bytes,
                            hip_stream);
}

gdr_status gdr_attention_backward_varlen(const gdr_attention_problem* p, int64_t rows, const int64_t* cu_seqlens,
                                         const void* q, const void* k, const void* v, const void* o, const float* lse,
                                         const void* dout, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                         void* hip_stream) {
  return attention_backward(p, rows, cu_seqlens, true, q, k, v, o, lse, dout, dq, dk, dv, ws, ws_bytes, hip_stream);
}

}  // extern "C"
