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
// accesses); the columns of an incomplete last vector are moved one by one.
#include "kda_device.h"
#include "kda_norm_launch.h"

namespace kda {
namespace {

constexpr int GATE_LINEAR = 0, GATE_SILU = 1;

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// N columns of a row from column c on, as fp32; columns past dim as 0.
template <typename T, int N>
__device__ __forceinline__ void load_cols(const T* row, int c, int dim, float (&f)[N]) {
  constexpr int VN = Vec<T>::N;
  if (c + N <= dim) {
#pragma unroll
    for (int b = 0; b < N; b += VN) {
      const typename Vec<T>::type v = *reinterpret_cast<const typename Vec<T>::type*>(row + c + b);
#pragma unroll
      for (int e = 0; e < VN; ++e) f[b + e] = to_f32((T)v[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = c + e < dim ? to_f32(row[c + e]) : 0.f;
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_cols(T* row, int c, int dim, const float (&f)[N]) {
  constexpr int VN = Vec<T>::N;
  if (c + N <= dim) {
#pragma unroll
    for (int b = 0; b < N; b += VN) {
      typename Vec<T>::type v;
#pragma unroll
      for (int e = 0; e < VN; ++e) v[e] = from_f32<T>(f[b + e]);
      *reinterpret_cast<typename Vec<T>::type*>(row + c + b) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < dim) row[c + e] = from_f32<T>(f[e]);
  }
}

__device__ __forceinline__ float gate_of(float z, int gate) {
  if (gate == GATE_LINEAR) return z;
  const float s = __builtin_amdgcn_rcpf(1.f + fast_exp2(-z * kLog2e));
  return gate == GATE_SILU ? z * s : s;
}

// The sum over a row's TPR threads, in every one of them.  Rows wider than a
// wave go through `red`; callers alternate between two such arrays, so that
// one barrier a reduction is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int off = 1; off < (TPR < 64 ? TPR : 64); off <<= 1) x += __shfl_xor(x, off, 64);
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
  float w[NI][N];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = (i * TPR + lane) * N;
    if (a.w) load_cols<float, N>(a.w, c, a.dim, w[i]);
    else {
#pragma unroll
      for (int e = 0; e < N; ++e) w[i][e] = 1.f;
    }
  }
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB, par ^= 1) {
    const int64_t row = row0 + sub;
    const int dim = row < a.rows ? a.dim : 0;  // a row past the end has no columns
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    const T* z = static_cast<const T*>(a.z) + row * a.zs;
    float f[NI][N], g[NI][N];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) load_cols<T, N>(x, (i * TPR + lane) * N, dim, f[i]);
    if (a.z) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        load_cols<T, N>(z, (i * TPR + lane) * N, dim, g[i]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          g[i][e] = gate_of(g[i][e], a.gate);
          if (a.gate_first) f[i][e] *= g[i][e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < N; ++e) ss += f[i][e] * f[i][e];
    ss = row_sum<TPR>(ss, red[par]);
    const float rs = __builtin_amdgcn_rsqf(ss * inv + a.eps);
    T* y = static_cast<T*>(a.y) + row * a.ys;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        f[i][e] = f[i][e] * rs * w[i][e];
        if (a.z && !a.gate_first) f[i][e] *= g[i][e];
      }
      store_cols<T, N>(y, (i * TPR + lane) * N, dim, f[i]);
    }
  }
}

template <typename T, typename TR, int TPR, int NI>
__global__ __launch_bounds__(threads_of<TPR>()) void block_norm_kernel(BlockNormArgs a) {
  constexpr int N = 16 / sizeof(T), NT = threads_of<TPR>(), RPB = NT / TPR;
  __shared__ float red[2][NT / 64];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.f / (float)a.dim;
  // scale c w_post and w_pre
  float wp[NI][N], wn[NI][N];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = (i * TPR + lane) * N;
#pragma unroll
    for (int e = 0; e < N; ++e) wp[i][e] = wn[i][e] = 1.f;
    if (a.w_post) load_cols<float, N>(a.w_post, c, a.dim, wp[i]);
    if (a.w_pre) load_cols<float, N>(a.w_pre, c, a.dim, wn[i]);
    if (a.c) {
      float f[N];
      load_cols<float, N>(a.c, c, a.dim, f);
#pragma unroll
      for (int e = 0; e < N; ++e) wp[i][e] *= f[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) wp[i][e] *= a.scale;
  }
  int par = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + sub;
    const int dim = row < a.rows ? a.dim : 0;
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    const T* z = static_cast<const T*>(a.z) + row * a.zs;
    const TR* r = static_cast<const TR*>(a.r) + row * a.rs;
    float f[NI][N], g[NI][N], res[NI][N];
#pragma unroll
    for (int i = 0; i < NI; ++i) load_cols<T, N>(x, (i * TPR + lane) * N, dim, f[i]);
#pragma unroll
    for (int i = 0; i < NI; ++i) load_cols<TR, N>(r, (i * TPR + lane) * N, dim, res[i]);
    if (a.z) {
#pragma unroll
      for (int i = 0; i < NI; ++i) load_cols<T, N>(z, (i * TPR + lane) * N, dim, g[i]);
    }
    float rs = 1.f;
    if (a.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) ss += f[i][e] * f[i][e];
      ss = row_sum<TPR>(ss, red[par]);
      par ^= 1;
      rs = __builtin_amdgcn_rsqf(ss * inv + a.eps);
    }
    float ss = 0.f;
    TR* ro = static_cast<TR*>(a.r_out) + row * a.ros;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float p = f[i][e] * rs * wp[i][e];
        if (a.z) p *= gate_of(g[i][e], a.gate);
        res[i][e] += p;
        ss += res[i][e] * res[i][e];
      }
      store_cols<TR, N>(ro, (i * TPR + lane) * N, dim, res[i]);
    }
    if (a.w_pre) {
      ss = row_sum<TPR>(ss, red[par]);
      par ^= 1;
      rs = __builtin_amdgcn_rsqf(ss * inv + a.eps);
      T* y = static_cast<T*>(a.y) + row * a.ys;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int e = 0; e < N; ++e) res[i][e] *= rs * wn[i][e];
        store_cols<T, N>(y, (i * TPR + lane) * N, dim, res[i]);
      }
    }
  }
}

// Threads per row and vectors per thread of a row of `nvec` vectors.
// (16,384 columns are 2,048 vectors of bf16 and 4,096 of fp32.)
template <typename T, typename L>
hipError_t dispatch(int nvec, const L& l) {
  if (nvec <= 8) return l.template run<8, 1>();
  if (nvec <= 16) return l.template run<16, 1>();
  if (nvec <= 32) return l.template run<32, 1>();
  if (nvec <= 64) return l.template run<64, 1>();
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
    gated_norm_kernel<T, TPR, NI><<<grid_of<TPR>(a.rows), threads_of<TPR>(), 0, stream>>>(a);
    return hipGetLastError();
  }
};

template <typename T, typename TR>
struct BlockLaunch {
  const BlockNormArgs& a;
  hipStream_t stream;
  template <int TPR, int NI>
  hipError_t run() const {
    block_norm_kernel<T, TR, TPR, NI><<<grid_of<TPR>(a.rows), threads_of<TPR>(), 0, stream>>>(a);
    return hipGetLastError();
  }
};

int vectors(int dim, bool bf) { return bf ? (dim + 7) / 8 : (dim + 3) / 4; }

}  // namespace

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
  if (a.bf16) return dispatch<bf16>(vectors(a.dim, true), GatedLaunch<bf16>{a, stream});
  return dispatch<float>(vectors(a.dim, false), GatedLaunch<float>{a, stream});
}

hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) {
  const int nv = vectors(a.dim, a.bf16);
  if (!a.bf16) return dispatch<float>(nv, BlockLaunch<float, float>{a, stream});
  if (a.res_bf16) return dispatch<bf16>(nv, BlockLaunch<bf16, bf16>{a, stream});
  return dispatch<bf16>(nv, BlockLaunch<bf16, float>{a, stream});
}

}  // namespace kda
