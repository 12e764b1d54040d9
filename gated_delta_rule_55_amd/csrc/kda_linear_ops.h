// kda_linear_ops.h -- device-side building blocks of linear attention: the
// 32x32 matrix-core step and its operands.
//
// Operand layout (gfx950, wave64), for A (32 x 16), B (16 x 32), D (32 x 32):
//   Lane l supplies row (l % 32) of A and column (l % 32) of B, and with
//   half = l / 32 the eight contraction indices of its half.  Which indices
//   those are is free as long as A and B agree.  D comes back with lane l
//   holding column l % 32 and, in register r, row (r % 4) + 8 (r / 4) + 4 half.
// A D tile of 32 rows is two contraction slices of the next product straight
// from registers: slice s takes registers 8s .. 8s + 7, so index e of half
// stands for D row 16s + 8 (e / 4) + 4 half + e % 4 ("D order").
#pragma once

#include "kda_device.h"

namespace kda {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// D += A B over 16 contraction indices.  bf16: one instruction; fp32: eight,
// each pairing index e of both halves.
__device__ __forceinline__ f32x16 mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma(f32x8 a, f32x8 b, f32x16 c) {
#pragma unroll
  for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
  return c;
}

// Row of a D tile held in register r of a lane's half.
__device__ __forceinline__ int d_row(int r, int half) { return (r & 3) + 8 * (r >> 2) + 4 * half; }

// Registers 8s .. 8s + 7 of a D tile as an operand in D order.
template <typename T>
__device__ __forceinline__ typename Frag<T>::type frag_of_d(const f32x16& d, int s) {
  typename Frag<T>::type f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = from_f32<T>(d[8 * s + e]);
  return f;
}

// The transpose of a 32-column, 16-row piece of an LDS tile [row][stride], in
// D order of its rows: lane l gets column l % 32 (or, with PERM, the column
// 16 ((l % 32) / 16) + 4 p(l % 16 / 4) + l % 4, p = 0, 2, 1, 3) of rows
// 4 half + e and 8 + 4 half + e.  p is what makes a D tile built with it as A
// hold eight consecutive columns in each lane's slice, so that the other
// operand of the next product is a plain 16-byte read.
// bf16: two transposing 8-byte LDS reads: in each group of 16 lanes, lane i
// addresses row i / 4, columns 4 (i % 4) .. + 3, and receives column i.
template <bool PERM>
__device__ __forceinline__ bf16x8 frag_t(const bf16* tile, int stride, int lane) {
  const int half = lane >> 5, i = lane & 15;
  int c4 = i & 3;
  if (PERM) c4 = (c4 >> 1) | ((c4 & 1) << 1);
  const bf16* p = tile + (4 * half + (i >> 2)) * stride + (lane & 16) + 4 * c4;
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)p);
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 8 * stride));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}
template <bool PERM>
__device__ __forceinline__ f32x8 frag_t(const float* tile, int stride, int lane) {
  const int half = lane >> 5, i = lane & 15;
  int c4 = i >> 2;
  if (PERM) c4 = (c4 >> 1) | ((c4 & 1) << 1);
  const float* p = tile + 4 * half * stride + (lane & 16) + 4 * c4 + (i & 3);
  f32x8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = p[(8 * (e >> 2) + (e & 3)) * stride];
  return f;
}

// x as a sum of three bf16 values, exactly (8 + 8 + 8 bits): each takes the
// upper half of what the ones before left.  (Where x is infinite the others
// are NaN, and so is the sum.)
__device__ __forceinline__ void split3(const f32x8& x, bf16x8& a, bf16x8& b, bf16x8& c) {
  unsigned int u[3][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float r = x[e];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      u[i][e] = __builtin_bit_cast(unsigned int, r);
      r -= __builtin_bit_cast(float, u[i][e] & 0xffff0000u);
    }
  }
  u32x4 p[3];
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) p[i][e] = __builtin_amdgcn_perm(u[i][2 * e + 1], u[i][2 * e], 0x07060302u);
  a = __builtin_bit_cast(bf16x8, p[0]);
  b = __builtin_bit_cast(bf16x8, p[1]);
  c = __builtin_bit_cast(bf16x8, p[2]);
}

// s, or NaN if any of the eight values is not finite: 0 times it is added.
__device__ __forceinline__ float add_nonfinite(bf16x8 f, float s) {
  const u32x4 u = __builtin_bit_cast(u32x4, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned int x = u[i];
    s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), bf16x2{(bf16)0.f, (bf16)0.f}, s, false);
  }
  return s;
}
__device__ __forceinline__ float add_nonfinite(f32x8 f, float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(f[i], 0.f, s);
  return s;
}
// (By value: a bit cast of a vector's element in place reads element 0.)
__device__ __forceinline__ bool finite1(float x) {
  return (__builtin_bit_cast(unsigned int, x) & 0x7f800000u) != 0x7f800000u;
}

}  // namespace kda
