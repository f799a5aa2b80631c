// The attention layer's operators: what their C entry points (gdr_attn_api.hip)
// and kernels (gdr_rotary.hip, gdr_cache.hip, gdr_attn.hip) share.  Shapes here
// are already validated, strides filled in (elements).
#pragma once

#include <gdr.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_internal.h"

namespace gdr {

// A paged cache; row offsets are counted in 16-byte units and fit 32 bits.
struct CacheView {
  int64_t pages, page_stride, token_stride, head_stride, table_row;
  int page_size, Hk, D, max_pages;
  const int32_t* table;
  const int64_t* lengths;
};

// Rotary positions, into rows (kc, vc null) or into a cache.
struct RotArgs {
  const void *q, *k, *v;
  const int64_t *pos, *cu;      // pos null: the place; cu null: T rows each
  const float* freq;
  void *qo, *ko;                // ko: rows, or the key cache
  void* vc;                     // the value cache
  CacheView cache;
  int64_t rows, B, T;
  int64_t q_row, k_row, v_row, qo_row, ko_row;
  int Hq, Hk, D;
  int section[4], axes, R;
  bool adjacent, cycled, back, append, io_bf16, out_bf16;
};
hipError_t launch_rotary(const RotArgs& a, hipStream_t st);

struct CacheAttnArgs {
  const void *q, *kc, *vc;
  void* o;
  float* lse;
  float* part;                  // workspace
  CacheView cache;
  int64_t B, q_row, max_len, window, sinks;
  int Hq;
  float scale;
  bool bf16, out_bf16;
};
size_t cache_attn_workspace(const CacheAttnArgs& a);  // looks at the sizes only
hipError_t launch_cache_attn(const CacheAttnArgs& a, hipStream_t st);

struct AttnArgs {
  const void *q, *k, *v, *out, *dout;  // out, dout: VJP
  const float* lse_in;
  const int64_t* cu;
  void *o, *dq, *dk, *dv;
  float* lse;
  char* ws;
  int64_t B, T, rows;
  int64_t q_row, k_row, v_row, window, sinks;
  int Hq, Hk, D;
  float scale;
  bool io_bf16, out_bf16;
};
hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t st);
size_t attn_bwd_workspace(const AttnArgs& a);
hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t st);

}  // namespace gdr
