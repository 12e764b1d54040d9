// kda_latent_ops.h -- device-side building blocks of latent attention: the
// 32 x 32 matrix step, a tile of rows in LDS, and the search that maps a
// workgroup to a sequence.
//
// Scores are formed transposed, S^T = K Q^T, so that a lane holds one query's
// scores and the softmax needs one exchange between the wave's halves.  D of the
// 32 x 32 step: lane l holds rows 8 (i / 4) + 4 (l / 32) + i % 4 (i = 0..15) of
// column l % 32.  Contraction slots: lane half h holds eight values e = 0..7 of
// a 16-wide slice; A and B only have to agree on which index (h, e) stands for:
//
//   columns of a row    8 h + e                        one 16-byte load in bf16
//   keys (values, P)    8 (e / 4) + 4 h + e % 4        what D leaves in registers,
//                                                      so P feeds the next product
#pragma once

#include "kda_device.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// D += A B over a 16-wide slice.  fp32: eight 32x32x2 steps, each pairing value
// e of both halves.
__device__ __forceinline__ f32x16 mma16(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma16(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// Row of element i of a D tile within its 32 rows, for lane half h.
__device__ __forceinline__ int row_of(int h, int i) { return 8 * (i >> 2) + 4 * h + (i & 3); }

// A tile of ROWS rows in LDS.  Rows are cut into column blocks of 128 bytes, each
// block a [ROWS][128 bytes] array whose 16-byte chunks are exchanged by the row's
// low three bits: eight rows' chunks of one column lie in different banks, and
// eight lanes that fetch a 128-byte line fill 128 consecutive bytes.
template <int ROWS>
__device__ __forceinline__ int tile_at(int row, int byte) {
  return (byte >> 7) * (ROWS * 128) + row * 128 + ((((byte >> 4) & 7) ^ (row & 7)) << 4) + (byte & 15);
}

// Columns c .. c + 7 of a row, as a fragment (c a multiple of 8).
template <int ROWS>
__device__ __forceinline__ bf16x8 tile_row8(const char* t, int row, int c, bf16) {
  return *reinterpret_cast<const bf16x8*>(t + tile_at<ROWS>(row, 2 * c));
}
template <int ROWS>
__device__ __forceinline__ f32x8 tile_row8(const char* t, int row, int c, float) {
  const f32x4 lo = *reinterpret_cast<const f32x4*>(t + tile_at<ROWS>(row, 4 * c));
  const f32x4 hi = *reinterpret_cast<const f32x4*>(t + tile_at<ROWS>(row, 4 * c + 16));
  return f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// The transposed fragment: column c0 + l % 32 of the 16 rows from row0, in the
// keys' order.  bf16: two transposing reads, in each of which 16 lanes fetch four
// rows' 16 columns (lane i four of row i / 4) and lane i receives column i of
// the four.
__device__ __forceinline__ s16x4 read_tr(const char* p) {
  typedef __attribute__((address_space(3))) s16x4* lds;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)p);
}
template <int ROWS>
__device__ __forceinline__ bf16x8 tile_col8(const char* t, int row0, int c0, int lane, bf16) {
  const int row = row0 + 4 * (lane >> 5) + ((lane & 15) >> 2);
  const int byte = 2 * (c0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3));
  const s16x4 lo = read_tr(t + tile_at<ROWS>(row, byte));
  const s16x4 hi = read_tr(t + tile_at<ROWS>(row + 8, byte));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}
template <int ROWS>
__device__ __forceinline__ f32x8 tile_col8(const char* t, int row0, int c0, int lane, float) {
  const int h = lane >> 5, byte = 4 * (c0 + (lane & 31));
  f32x8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    f[e] = *reinterpret_cast<const float*>(t + tile_at<ROWS>(row0 + 8 * (e >> 2) + 4 * h + (e & 3), byte));
  return f;
}

// Values that are not finite, in rows that some of a tile's queries see and
// others do not: a weight of 0 would turn them into NaN for all.  They are taken
// out of the fragment and counted by kind in a product with the queries' sight
// instead (1 for +inf, 2^10 for -inf, 2^20 for NaN; a tile's 64 keys keep the
// sums apart), which add_special gives back to the queries that do see them.
template <typename F>
__device__ __forceinline__ void split_special(F& v, F& kind) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float x = (float)v[e];
    const bool finite = __builtin_isfinite(x);
    kind[e] = finite ? 0.f : (x != x ? 1048576.f : (x > 0.f ? 1.f : 1024.f));
    if (!finite) v[e] = 0.f;
  }
}
__device__ __forceinline__ float add_special(float acc, float kinds) {
  if (kinds == 0.f) return acc;
  const float inf = __builtin_inff();
  if (kinds >= 1048576.f) return __builtin_nanf("");
  const bool neg = kinds >= 1024.f;
  const bool pos = kinds != 1024.f * __builtin_floorf(kinds * (1.f / 1024.f));
  if (pos) acc += inf;
  if (neg) acc -= inf;
  return acc;
}

// 16 bytes from each lane's place in the buffer to 1,024 consecutive bytes of LDS,
// without passing through registers; a lane whose place lies outside the buffer
// writes 0.  `at` is the wave's own part of LDS.  What is fetched is there once the
// wave has waited (fetched()).  The compiler orders LDS reads behind a fetch into
// the same array only, so what is read while a fetch is under way is an array of its
// own.
__device__ __forceinline__ void fetch16(__amdgpu_buffer_rsrc_t r, int place, int uniform, char* at) {
  typedef __attribute__((address_space(3))) void* lds;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds)at, 16, place, uniform, 0, 0);
}
// Waits for this wave's fetches and LDS accesses, then for the workgroup's other waves.
__device__ __forceinline__ void fetched() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Values of the other half of the wave (lane l ^ 32).
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// cu[n], or n where there is no table (one token each), clamped to [0, total].
__device__ __forceinline__ int seq_start(const int32_t* cu, int n, int total) {
  const int c = cu ? cu[n] : n;
  return c < 0 ? 0 : (c > total ? total : c);
}

// The last n of 0 .. count - 1 for which before(n) holds, where it holds for a first
// stretch of them (0 where it holds for none).  All lanes of the wave search
// together, 64 places at a time; whatever before() answers, the result is in range.
template <typename Before>
__device__ __forceinline__ int find_last(int count, Before before) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = count;  // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len - 1) / 64 + 1, at = lane * step;
    const int c = max(__popcll(__ballot(lane <= (len - 1) / step && before(lo + at))), 1) - 1;
    lo += c * step;
    len = min(step, len - c * step);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// A sequence's tokens, `per` rows each, in blocks of B rows: numbered from here on,
// the blocks of two sequences never share a number, and no sequence needs the
// lengths of those before it for its own.  A number may belong to none.
template <int B>
__device__ __forceinline__ int64_t first_block(int start, int per, int n) {
  return (int64_t)start * per / B + n;
}
template <int B>
__device__ __forceinline__ int find_sequence(const int32_t* cu, int n_seqs, int total, int per, int64_t block) {
  return find_last(n_seqs, [=](int n) { return first_block<B>(seq_start(cu, n, total), per, n) <= block; });
}

}  // namespace kda
