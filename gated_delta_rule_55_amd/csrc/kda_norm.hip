// kda_norm.hip -- row norms fused with what stands around them in a layer:
// the gated output norm of the recurrence (kda_gated_norm) and the norms
// before and after a block with its gate, scale and residual (kda_block_norm).
//
// Both are one pass over their rows: TPR threads hold a row in registers, NI
// vectors of 16 bytes each, so every operand is read once and every result
// written once, whatever is fused.  Sums of squares are fp32, reduced over
// lanes and, for rows wider than a wave, through LDS.  A workgroup walks
// several rows and keeps its columns' weights in registers.  Vectors need
// only their elements' alignment (the hardware takes unaligned 16-byte
// accesses).
//
// Bound by the memory: 1 M rows of 128 in bf16 with a gate, 805 MB, 147 us
// (5.5 TB/s, above a copy's 4.75: two reads to a write); 32,768 rows of 4,096
// around a block with every option, 1.34 GB, 245 us (5.5 TB/s), as a plain add and
// norm, 1.07 GB, 187 us (5.7).  In fp32 half as many rows are the same bytes: 159
// us for the gate, 251 and 195 around a block.  Rows of 4,097,
// whose vectors are not aligned, run at 4.1 to 4.9 TB/s.
#include "kda_device.h"
#include "kda_enqueue.h"
#include "kda_norm_launch.h"

namespace kda {
namespace {

constexpr int GATE_LINEAR = 0, GATE_SILU = 1;

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// A thread's columns of a row: NI vectors of N, the i-th being vector
// i TPR + lane of the row's whole vectors, and one column of the row's rest
// (fewer than N columns, one each for the first lanes; N <= TPR).  What lies
// past the row's end is 0 and is not stored.
template <int NI, int N>
struct Columns {
  float v[NI][N];
  float rest;

  template <typename F>
  __device__ __forceinline__ void each(F f) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) f(v[i][e]);
    f(rest);
  }
  // f(this value, o's value of the same column)
  template <typename F>
  __device__ __forceinline__ void with(const Columns& o, F f) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) f(v[i][e], o.v[i][e]);
    f(rest, o.rest);
  }
  __device__ __forceinline__ void fill(float x) {
    each([&](float& y) { y = x; });
  }
  __device__ __forceinline__ float squares() {
    float s = 0.f;
    each([&](float& x) { s += x * x; });
    return s;
  }

  template <int TPR, typename T>
  __device__ __forceinline__ void load(const T* row, int lane, int dim) {
    constexpr int VN = Vec<T>::N;
    const int whole = dim / N;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * TPR + lane;
#pragma unroll
      for (int e = 0; e < N; ++e) v[i][e] = 0.f;
      if (c < whole) {
#pragma unroll
        for (int b = 0; b < N; b += VN) {
          const typename Vec<T>::type x = *reinterpret_cast<const typename Vec<T>::type*>(row + c * N + b);
#pragma unroll
          for (int e = 0; e < VN; ++e) v[i][b + e] = to_f32((T)x[e]);
        }
      }
    }
    rest = 0.f;
    if (whole * N + lane < dim) rest = to_f32(row[whole * N + lane]);
  }
  template <int TPR, typename T>
  __device__ __forceinline__ void store(T* row, int lane, int dim) const {
    constexpr int VN = Vec<T>::N;
    const int whole = dim / N;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * TPR + lane;
      if (c < whole) {
#pragma unroll
        for (int b = 0; b < N; b += VN) {
          typename Vec<T>::type x;
#pragma unroll
          for (int e = 0; e < VN; ++e) x[e] = from_f32<T>(v[i][b + e]);
          *reinterpret_cast<typename Vec<T>::type*>(row + c * N + b) = x;
        }
      }
    }
    if (whole * N + lane < dim) row[whole * N + lane] = from_f32<T>(rest);
  }
};

__device__ __forceinline__ float gate_of(float z, int gate) {
  if (gate == GATE_LINEAR) return z;
  const float s = __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
  return gate == GATE_SILU ? z * s : s;
}

// x plus that of the lane which differs in this one bit (OFF 1, 2, 16 or 32), or
// of one whose group of OFF lanes does (4 and 8: the lane mirrored in 8 and in
// 16), which is the same once x is equal within groups.
template <int OFF>
__device__ __forceinline__ float plus_lane(float x) {
  const int b = __builtin_bit_cast(int, x);
  if constexpr (OFF == 32 || OFF == 16) {  // the swap of x with itself leaves one half in each
    const auto pair = OFF == 32 ? __builtin_amdgcn_permlane32_swap(b, b, false, false)
                                : __builtin_amdgcn_permlane16_swap(b, b, false, false);
    const int lo = pair[0], hi = pair[1];
    return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
  } else {
    constexpr int ctrl = OFF == 1 ? 0xB1 : OFF == 2 ? 0x4E : OFF == 4 ? 0x141 : 0x140;
    return x + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(b, ctrl, 0xF, 0xF, true));
  }
}

// The sum over a row's TPR threads, in every one of them.  Rows wider than a
// wave go through `red`; callers alternate between two such arrays, so that
// one barrier a reduction is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
  x = plus_lane<1>(x);
  x = plus_lane<2>(x);
  x = plus_lane<4>(x);
  if constexpr (TPR > 8) x = plus_lane<8>(x);
  if constexpr (TPR > 16) x = plus_lane<16>(x);
  if constexpr (TPR > 32) x = plus_lane<32>(x);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = x;
    __syncthreads();
    const float* mine = red + wave / W * W;
    x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += mine[i];
  }
  return x;
}

template <int TPR>
constexpr int threads_of() {
  return TPR < 256 ? 256 : TPR;
}

template <typename T, int TPR, int NI>
__global__ __launch_bounds__(threads_of<TPR>()) void gated_norm_kernel(GatedNormArgs a) {
  constexpr int N = 16 / sizeof(T), NT = threads_of<TPR>(), RPB = NT / TPR;
  __shared__ float red[2][NT / 64];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.f / (float)a.dim;
  Columns<NI, N> w, f, g;
  w.fill(1.f);
  if (a.w) w.template load<TPR>(a.w, lane, a.dim);
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, par ^= 1) {
    const int64_t row = row0 + sub;
    const int dim = row < a.rows ? a.dim : 0;  // a row past the end has no columns
    f.template load<TPR>(static_cast<const T*>(a.x) + row * a.xs, lane, dim);
    if (a.z) {
      g.template load<TPR>(static_cast<const T*>(a.z) + row * a.zs, lane, dim);
      g.each([&](float& z) { z = gate_of(z, a.gate); });
      if (a.gate_first) f.with(g, [](float& x, float z) { x *= z; });
    }
    const float ss = row_sum<TPR>(f.squares(), red[par]);
    const float rs = __builtin_amdgcn_rsqf(ss * inv + a.eps);
    f.with(w, [&](float& x, float y) { x *= rs * y; });
    if (a.z && !a.gate_first) f.with(g, [](float& x, float z) { x *= z; });
    f.template store<TPR>(static_cast<T*>(a.y) + row * a.ys, lane, dim);
  }
}

template <typename T, typename TR, int TPR, int NI>
__global__ __launch_bounds__(threads_of<TPR>()) void block_norm_kernel(BlockNormArgs a) {
  constexpr int N = 16 / sizeof(T), NT = threads_of<TPR>(), RPB = NT / TPR;
  __shared__ float red[2][NT / 64];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.f / (float)a.dim;
  Columns<NI, N> wp, wn, f, g, r;  // wp: scale c w_post
  wp.fill(1.f);
  if (a.w_post) wp.template load<TPR>(a.w_post, lane, a.dim);
  if (a.c) {
    f.template load<TPR>(a.c, lane, a.dim);
    wp.with(f, [](float& x, float c) { x *= c; });
  }
  wp.each([&](float& x) { x *= a.scale; });
  wn.fill(1.f);
  if (a.w_pre) wn.template load<TPR>(a.w_pre, lane, a.dim);
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + sub;
    const int dim = row < a.rows ? a.dim : 0;
    f.template load<TPR>(static_cast<const T*>(a.x) + row * a.xs, lane, dim);
    r.template load<TPR>(static_cast<const TR*>(a.r) + row * a.rs, lane, dim);
    if (a.z) g.template load<TPR>(static_cast<const T*>(a.z) + row * a.zs, lane, dim);
    float rs = 1.f;
    if (a.w_post) {
      const float ss = row_sum<TPR>(f.squares(), red[par]);
      par ^= 1;
      rs = __builtin_amdgcn_rsqf(ss * inv + a.eps);
    }
    f.with(wp, [&](float& x, float y) { x *= rs * y; });
    if (a.z) f.with(g, [&](float& x, float z) { x *= gate_of(z, a.gate); });
    r.with(f, [](float& x, float p) { x += p; });
    r.template store<TPR>(static_cast<TR*>(a.r_out) + row * a.ros, lane, dim);
    if (a.w_pre) {
      const float ss = row_sum<TPR>(r.squares(), red[par]);
      par ^= 1;
      rs = __builtin_amdgcn_rsqf(ss * inv + a.eps);
      r.with(wn, [&](float& x, float y) { x *= rs * y; });
      r.template store<TPR>(static_cast<T*>(a.y) + row * a.ys, lane, dim);
    }
  }
}

// Threads per row and vectors per thread of a row of `nvec` vectors: at most two
// vectors each (a block norm holds five operands of each in registers), four
// where 1,024 threads do not go round otherwise.  (16,384 columns are 2,048
// vectors of bf16 and 4,096 of fp32.)  Up to 512 rows leave the chip half empty
// and the time is one row's: then one vector each, up to 512 threads (rows of
// 4,096 in bf16 with a gate, and around a block with every option and an fp32
// residual, one vector against two: 64 rows 3.3 against 3.7 us and 4.4 against
// 4.8, 512 rows 4.4 against 4.6 and 7.2 against 7.5; 1,024 rows 6.6 against 7.1
// and 11.9 against 11.3).
template <typename T, typename L>
hipError_t dispatch(int64_t rows, int nvec, const L& l) {
  if (nvec <= 8) return l.template run<8, 1>();
  if (nvec <= 16) return l.template run<16, 1>();
  if (nvec <= 32) return l.template run<32, 1>();
  if (nvec <= 64) return l.template run<64, 1>();
  if (rows <= 512 && nvec <= 512) {
    if (nvec <= 128) return l.template run<128, 1>();
    if (nvec <= 256) return l.template run<256, 1>();
    return l.template run<512, 1>();
  }
  if (nvec <= 128) return l.template run<64, 2>();
  if (nvec <= 256) return l.template run<128, 2>();
  if (nvec <= 512) return l.template run<256, 2>();
  if (nvec <= 1024) return l.template run<512, 2>();
  if constexpr (sizeof(T) == 4) {
    if (nvec > 2048) return l.template run<1024, 4>();
  }
  return l.template run<1024, 2>();
}

// Workgroups: 2048 threads on each of 256 CUs, rows beyond that in a loop.
template <int TPR>
unsigned grid_of(int64_t rows) {
  constexpr int NT = threads_of<TPR>(), RPB = NT / TPR;
  const int64_t need = (rows + RPB - 1) / RPB, most = 256 * (2048 / NT);
  return (unsigned)(need < most ? need : most);
}

template <typename T>
struct GatedLaunch {
  const GatedNormArgs& a;
  hipStream_t stream;
  template <int TPR, int NI>
  hipError_t run() const {
    return enqueue(gated_norm_kernel<T, TPR, NI>, grid_of<TPR>(a.rows), threads_of<TPR>(), stream, a);
  }
};

template <typename T, typename TR>
struct BlockLaunch {
  const BlockNormArgs& a;
  hipStream_t stream;
  template <int TPR, int NI>
  hipError_t run() const {
    return enqueue(block_norm_kernel<T, TR, TPR, NI>, grid_of<TPR>(a.rows), threads_of<TPR>(), stream, a);
  }
};

// Whole vectors of a row; its rest goes one column a thread.
int vectors(int dim, bool bf) { return bf ? dim / 8 : dim / 4; }

}  // namespace

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
  if (a.bf16) return dispatch<bf16>(a.rows, vectors(a.dim, true), GatedLaunch<bf16>{a, stream});
  return dispatch<float>(a.rows, vectors(a.dim, false), GatedLaunch<float>{a, stream});
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  const int nv = vectors(a.dim, a.bf16);
  if (!a.bf16) return dispatch<float>(a.rows, nv, BlockLaunch<float, float>{a, stream});
  if (a.res_bf16) return dispatch<bf16>(a.rows, nv, BlockLaunch<bf16, bf16>{a, stream});
  return dispatch<bf16>(a.rows, nv, BlockLaunch<bf16, float>{a, stream});
}

}  // namespace kda
