// kda_latent_launch.h -- internal interface between the C ABI of latent
// attention (kda_latent_abi.cpp) and its launchers.  Arguments here are
// already validated; strides are resolved, in elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct LatentPrefillArgs {
  bool bf16;
  int n_seqs, n_heads, dn, dr, dv;
  int q_total, k_total;
  float scale;
  const void *q, *k, *pe, *v;
  void* o;
  int64_t q_stride, k_stride, k_head, pe_stride, v_stride, v_head, o_stride;
  const int32_t* cu;    // NULL: one sequence
  const int32_t* cu_k;  // NULL: cu
};

// The tables of a paged cache.
struct LatentPages {
  int page_size, max_pages, n_pages;
  uint32_t page_factor;  // j / page_size = j page_factor >> page_shift for 0 <= j < 2^31:
  int page_shift;        // ceil(2^shift / size), shift = 31 + ceil(log2 size)
  int64_t page_stride, row_stride;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;  // NULL: one token per sequence
  int n_seqs;
  int t_total;
};

struct LatentAttendArgs {
  bool bf16;
  int n_heads, dc, dr;
  float scale;
  const void *q, *cache;
  void* o;
  int64_t q_stride, o_stride;
  LatentPages pages;
};

struct LatentAppendArgs {
  bool bf16;
  int dc, dr;
  bool interleaved;
  float eps, magnitude;
  const void *latent, *pe;
  void *cache, *rows;
  int64_t latent_stride, pe_stride, rows_stride;
  const float* weight;
  const double* frequencies;
  LatentPages pages;
};

struct RotaryArgs {
  bool bf16;
  int n_heads, dim;
  bool interleaved;
  float magnitude;
  int t_total;
  const void* x;
  void* y;
  int64_t x_stride, x_head, y_stride, y_head;
  const int32_t* positions;
  const double* frequencies;
};

// Workgroups per head of a prefill: query blocks that a batch of q_total tokens
// in n_seqs sequences has at most.
constexpr int kLatentQueryBlock = 128;
inline int64_t latent_query_blocks(int64_t q_total, int64_t n_seqs) { return q_total / kLatentQueryBlock + n_seqs; }
size_t latent_prefill_workspace_bytes(const LatentPrefillArgs& a);
hipError_t launch_latent_prefill(const LatentPrefillArgs& a, void* workspace, hipStream_t stream);

size_t latent_workspace_bytes(const LatentAttendArgs& a);
hipError_t launch_latent_attend(const LatentAttendArgs& a, void* workspace, hipStream_t stream);

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t stream);
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);

}  // namespace kda
