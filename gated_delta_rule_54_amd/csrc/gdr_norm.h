// Group norm of the heads' outputs: what its C entry points
// (gdr_linear_api.hip) and kernels (gdr_norm.hip) share.
#pragma once

#include <gdr.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdr_internal.h"

namespace gdr {

struct NormArgs {
  const void *x, *z, *dy;  // z: null without a gate; dy: backward
  const float *w, *b;      // null: ones, zeros
  void *y, *dx, *dz;
  float *dw, *db;          // null: not wanted
  float* part;             // backward workspace
  int64_t rows, x_row, z_row;  // rows; elements between rows of x and z
  int G, D;
  float eps;
  bool io_bf16, out_bf16, center, silu, shared;
};

hipError_t launch_norm_fwd(const NormArgs& a, hipStream_t st);
size_t norm_bwd_workspace(const NormArgs& a);  // looks at the sizes and flags only
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t st);

}  // namespace gdr
