// kda_linear_launch.h -- internal interface between the C ABI of linear
// attention (kda_linear_abi.cpp) and its launchers.  Arguments here are
// already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct LinearPrefillArgs {
  bool bf16;
  bool state_bf16;
  bool decay_head;  // g is [H], else [T, H]
  int n_seqs, n_heads, kheads, dk, dv;
  int64_t t_total;
  float scale;
  const void *q, *k, *v;
  const float* g;
  void* o;
  int64_t q_stride, k_stride, v_stride, o_stride;  // elements, resolved
  const void* h0;
  void* ht;
  const int32_t* cu_seqlens;  // may be NULL when n_seqs == 1
  const int32_t* slots;
  int n_slots;
};

struct LinearDecodeArgs {
  bool bf16;
  bool state_bf16;
  bool decay_head;
  int n_seqs, n_heads, kheads, dk, dv;
  float scale;
  void* state;
  const void *q, *k, *v;
  const float* g;
  void* o;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const int32_t* slots;
  int n_slots;
};

// Tokens per segment: a sequence longer than this is split (kda_linear.hip).
int64_t linear_segment(int64_t t_total, int n_seqs, int n_heads, int dv, bool bf16);
// Workgroups per head of a segmented launch: at most t_total / seg + n_seqs
// segments exist.
inline int64_t linear_segments(int64_t t_total, int n_seqs, int64_t seg) {
  return t_total / seg + n_seqs;
}
size_t linear_workspace_bytes(const LinearPrefillArgs& a);
hipError_t launch_linear_prefill(const LinearPrefillArgs& a, void* workspace, hipStream_t stream);
hipError_t launch_linear_decode(const LinearDecodeArgs& a, hipStream_t stream);

}  // namespace kda
