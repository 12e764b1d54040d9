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
#include "kda_latent_launch.h"

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
// block a [ROWS][128 bytes] array whose 16-byte chunks are exchanged by a number of the
// row: eight rows' chunks of one column lie in different banks, and so do 64 bytes of
// rows r and r + 2 (banks repeat after 256 bytes, two rows), which a transposing read
// fetches together.
__device__ __forceinline__ int row_swap(int row) { return (row & 1) | (row & 2) << 1 | (row & 4) >> 1; }
template <int ROWS>
__device__ __forceinline__ int tile_at(int row, int byte) {
  return (byte >> 7) * (ROWS * 128) + row * 128 + ((((byte >> 4) & 7) ^ row_swap(row)) << 4) + (byte & 15);
}

// A value that the compiler keeps in a register as it is: an address that constants
// are added to (they go into the instructions) instead of one address for each.
__device__ __forceinline__ int kept(int x) {
  asm("" : "+v"(x));
  return x;
}

// Fragments of a tile's rows: columns 8 x .. 8 x + 7 of every slice of STEP columns,
// for the lane's row and x.
template <typename T, int ROWS, int STEP>
struct RowFrags {
  static constexpr int N = 128 / (STEP * sizeof(T)), HALVES = sizeof(T) / 2;
  int at[N][HALVES];
  __device__ __forceinline__ RowFrags(int row, int x) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int f = 0; f < HALVES; ++f) at[n][f] = kept(tile_at<ROWS>(row, (STEP * n + 8 * x) * (int)sizeof(T) + 16 * f));
  }
  // slice s, `below` rows (a multiple of 8) below the lane's
  __device__ __forceinline__ typename Frag<T>::type load(const char* tile, int s, int below) const {
    const char* p = tile + (s / N) * (ROWS * 128) + below * 128;
    typename Frag<T>::type f;
    if constexpr (HALVES == 1) {
      f = *reinterpret_cast<const bf16x8*>(p + at[s % N][0]);
    } else {
      const f32x4 lo = *reinterpret_cast<const f32x4*>(p + at[s % N][0]);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(p + at[s % N][1]);
      f = f32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    return f;
  }
};

// Transposed fragments: column c0 + 32 d + lane % 32 of 16 rows, in the keys' order (c0
// a multiple of 64, or of 32 where d is 0).  bf16: two transposing reads, in each of
// which 16 lanes fetch four rows' 16 columns (lane i four of row i / 4) and lane i
// receives column i of the four.
__device__ __forceinline__ s16x4 read_tr(const char* p) {
  typedef __attribute__((address_space(3))) s16x4* lds;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)p);
}
template <typename T, int ROWS>
struct ColFrags {
  static constexpr int N = sizeof(T) == 2 ? 2 : 4;
  int at[N];
  __device__ __forceinline__ ColFrags(int c0, int lane) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if constexpr (sizeof(T) == 2)
        at[n] = tile_at<ROWS>(4 * (lane >> 5) + ((lane & 15) >> 2), 2 * (c0 + 32 * n + 16 * ((lane >> 4) & 1) + 4 * (lane & 3)));
      else
        at[n] = tile_at<ROWS>(4 * (lane >> 5) + n, 4 * (c0 + (lane & 31)));
      at[n] = kept(at[n]);
    }
  }
  // the 16 rows from row0 (a multiple of 16); d may be a variable (no register is indexed)
  __device__ __forceinline__ typename Frag<T>::type load(const char* tile, int row0, int d) const {
    typename Frag<T>::type f;
    if constexpr (sizeof(T) == 2) {
      const int first = at[0], second = at[1];
      const char* p = tile + (d / 2) * (ROWS * 128) + row0 * 128 + (d % 2 ? second : first);
      const s16x4 lo = read_tr(p), hi = read_tr(p + 8 * 128);
      typedef short s16x8 __attribute__((ext_vector_type(8)));
      f = __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        f[e] = *reinterpret_cast<const float*>(tile + d * (ROWS * 128) + (row0 + 8 * (e >> 2)) * 128 + at[e & 3]);
    }
    return f;
  }
};

// N matrix steps whose operands come from LDS, in groups of G: a group's operands are
// read while the group before runs.  (Left to itself the compiler reads each operand
// right before its step, where registers are short.)  load(i) answers step i's operand,
// step(i, operand) runs it, and between(g) is other work for behind group g's steps.
// `now` holds the first group's operands.
template <typename F, int N, int G, typename Load, typename Step, typename Between>
__device__ __forceinline__ void pipelined_from(F (&now)[G], Load load, Step step, Between between) {
  F next[G];
#pragma unroll
  for (int g = 0; g < N; g += G) {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (g + G + i < N) next[i] = load(g + G + i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (g + i < N) step(g + i, now[i]);
    between(g / G);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < G; ++i) now[i] = next[i];
  }
}
template <typename F, int N, int G, typename Load, typename Step, typename Between>
__device__ __forceinline__ void pipelined(Load load, Step step, Between between) {
  F now[G];
#pragma unroll
  for (int i = 0; i < G; ++i) now[i] = load(i);
  pipelined_from<F, N, G>(now, load, step, between);
}
template <typename F, int N, int G, typename Load, typename Step>
__device__ __forceinline__ void pipelined(Load load, Step step) {
  pipelined<F, N, G>(load, step, [](int) {});
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
    const uint32_t bits = __builtin_bit_cast(uint32_t, x);
    const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
    const float which = (bits & 0x7fffffu) ? 1048576.f : (bits >> 31) ? 1024.f : 1.f;
    kind[e] = finite ? 0.f : which;
    v[e] = finite ? x : 0.f;
  }
}
__device__ __forceinline__ float add_special(float acc, float kinds) {
  const float inf = __builtin_inff();
  const bool nan = kinds >= 1048576.f, neg = kinds >= 1024.f;
  const bool pos = kinds != 1024.f * __builtin_floorf(kinds * (1.f / 1024.f));
  acc += pos || nan ? inf : 0.f;
  acc -= neg ? inf : 0.f;  // both kinds, and NaN's own: inf - inf
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
// The same from a pointer of each lane's own.
__device__ __forceinline__ void fetch16(const char* from, char* at) {
  typedef __attribute__((address_space(3))) void* lds;
  typedef const __attribute__((address_space(1))) void* global;
  __builtin_amdgcn_global_load_lds((global)from, (lds)at, 16, 0, 0);
}
// p + 128.  (Written out: the compiler adds to 64-bit addresses from scalar registers, a
// pair for each multiple of 128, and runs out of them.)
__device__ __forceinline__ const char* next_line(const char* p) {
  uint32_t lo = (uint32_t)(uintptr_t)p, hi = (uint32_t)((uintptr_t)p >> 32);
  asm("v_add_co_u32 %0, vcc, 0x80, %0\n\tv_addc_co_u32 %1, vcc, 0, %1, vcc" : "+v"(lo), "+v"(hi) : : "vcc");
  return reinterpret_cast<const char*>((uintptr_t)hi << 32 | lo);
}
// Waits for this wave's LDS accesses, then for the workgroup's other waves.  (Fetches
// stay under way, which __syncthreads would wait for.)
__device__ __forceinline__ void exchanged() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// The same, and for this wave's fetches.
__device__ __forceinline__ void fetched() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Values of the other half of the wave (lane l ^ 32).
__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// The larger of the values of lanes l and l ^ 32, l and l ^ 16, in both.  (The swaps exchange the
// halves, or neighbouring sixteens, of two registers, without the way through LDS that a shuffle
// takes.)
__device__ __forceinline__ float larger_of(__attribute__((ext_vector_type(2))) unsigned x) {
  return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
__device__ __forceinline__ float max_halves(float x) {
  return larger_of(__builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false));
}
__device__ __forceinline__ float max_sixteens(float x) {
  return larger_of(__builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false));
}

// The wave of this thread in its workgroup, as a scalar.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// A value that all lanes have, as a scalar.  What is read from LDS counts as different
// in each lane otherwise, and a branch on it as one that lanes take by themselves: the
// kernels here have none of those where registers are full, since copies that the
// compiler (AMD clang 22 of ROCm 7.2) makes behind such a branch, to free registers, have
// missed lanes.  tests/test_latent_codegen_host.py looks for both in what it made.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
  return (int64_t)((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32 | (uint32_t)uniform((int)x));
}

// Ends a variant's code in a way of its own: the compiler would share the ends of two
// variants of a function, and move all their registers to where both have them.
template <bool VARIANT>
__device__ __forceinline__ void end_of_variant() {
  asm volatile("; variant %0" : : "n"(VARIANT));
}

// Four neighbouring values of an output row; none where `off` is kBufferOff.
__device__ __forceinline__ void store4(bf16x4 v, __amdgpu_buffer_rsrc_t r, int off) {
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, v), r, off, 0, 0);
}
__device__ __forceinline__ void store4(f32x4 v, __amdgpu_buffer_rsrc_t r, int off) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 0);
}

// The page of position j of a sequence (0 <= j < 2^31), and j's row there.
__device__ __forceinline__ int page_of(const LatentPages& g, int j) {
  return (int)((uint64_t)(uint32_t)j * g.page_factor >> g.page_shift);
}
__device__ __forceinline__ int row_in_page(const LatentPages& g, int j, int page) { return j - page * g.page_size; }

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
