// kda_norm_launch.h -- internal interface between the C ABI of the norms
// (kda_norm_abi.cpp) and their launchers.  Arguments here are already
// validated; strides are resolved.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct GatedNormArgs {
  bool bf16;
  int dim, gate;
  bool gate_first;
  float eps;
  int64_t rows;
  const void* x;
  const float* w;
  const void* z;
  void* y;
  int64_t xs, zs, ys;
};

struct BlockNormArgs {
  bool bf16, res_bf16;
  int dim, gate;
  float eps, scale;
  int64_t rows;
  const void *x, *r;
  const float *w_post, *w_pre, *c;
  const void* z;
  void *r_out, *y;
  int64_t xs, rs, zs, ros, ys;
};

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream);
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream);

}  // namespace kda
