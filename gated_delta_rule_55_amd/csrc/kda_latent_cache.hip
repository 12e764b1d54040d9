// kda_latent_cache.hip -- rows of the paged latent cache (kda_latent_append) and
// the rotation of positional parts (kda_rotary).
//
// The angle position x frequency is formed in fp64 in turns and reduced to
// [-1/2, 1/2] there, so that its sine and cosine (fp32, sincospi) are as exact
// at position 10^6 as at 1.  Both are bound by the memory; the angles are shared
// by all heads of a token.  Measured, bf16: 32,768 rows of 512 + 64 appended in 16.5 us (4.6
// TB/s), 32,768 tokens of 32 heads of 64 turned in 55 us (4.9 TB/s, a copy's rate);
// 64 tokens of either take 4.4 us, which is the call: the kernels take 3.5 and 4.4.
#include "kda_enqueue.h"
#include "kda_latent_launch.h"
#include "kda_latent_ops.h"

namespace kda {
namespace {

constexpr double kInvTwoPi = 0.15915494309189533577;

__device__ __forceinline__ void turn_of(double position, double frequency, float magnitude, float& cosine, float& sine) {
  const double turns = position * (frequency * kInvTwoPi);
  const float part = (float)(2.0 * (turns - __builtin_rint(turns)));  // half turns, in [-1, 1]
  float s, c;
  sincospif(part, &s, &c);
  cosine = magnitude * c;
  sine = magnitude * s;
}

// -- append: one wave per token -----------------------------------------------------------

constexpr int APPEND_TOKENS = 4;  // per workgroup

template <typename T, int DC, int DR>
__global__ __launch_bounds__(64 * APPEND_TOKENS) void latent_append_kernel(LatentAppendArgs a) {
  constexpr int E = 16 / sizeof(T), CHUNKS = DC / E, NI = (CHUNKS + 63) / 64;
  typedef T VecT __attribute__((ext_vector_type(E)));
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * APPEND_TOKENS + (threadIdx.x >> 6);
  const LatentPages& g = a.pages;
  if (t >= g.t_total) return;
  int n = (int)t, back = 1;  // the sequence, and the token's place from its end
  if (g.cu) {
    n = find_last(g.n_seqs, [&](int i) { return seq_start(g.cu, i, g.t_total) <= t; });
    const int start = seq_start(g.cu, n, g.t_total), end = seq_start(g.cu, n + 1, g.t_total);
    if (t < start || t >= end) return;
    back = end - (int)t;
  }
  const int64_t at = (int64_t)g.lens[n] - back;
  const T* lat = static_cast<const T*>(a.latent) + t * a.latent_stride;
  const T* pe = static_cast<const T*>(a.pe) + t * a.pe_stride;
  VecT x[NI];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int v = 64 * i + lane;
    if (v < CHUNKS) {
      x[i] = *reinterpret_cast<const VecT*>(lat + v * E);
#pragma unroll
      for (int e = 0; e < E; ++e) ss += (float)x[i][e] * (float)x[i][e];
    }
  }
  // the positional part: pair i of the rotation in lane i
  float pa = 0.f, pb = 0.f;
  const int ia = a.interleaved ? 2 * lane : lane, ib = a.interleaved ? 2 * lane + 1 : lane + DR / 2;
  if (lane < DR / 2) {
    pa = (float)pe[ia];
    pb = (float)pe[ib];
    if (a.frequencies) {
      float c, s;
      turn_of((double)at, a.frequencies[lane], a.magnitude, c, s);
      const float y = pa * c - pb * s;
      pb = pb * c + pa * s;
      pa = y;
    }
  }
  if (a.weight) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) ss += __shfl_xor(ss, d);
    const float r = 1.f / __builtin_sqrtf(ss * (1.f / DC) + a.eps);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = 64 * i + lane;
      if (v < CHUNKS)
#pragma unroll
        for (int e = 0; e < E; ++e) x[i][e] = from_f32<T>((float)x[i][e] * r * a.weight[v * E + e]);
    }
  }
  T* row[2] = {a.rows ? static_cast<T*>(a.rows) + t * a.rows_stride : nullptr, nullptr};
  if (at >= 0 && at < (int64_t)g.max_pages * g.page_size) {
    const int place = page_of(g, (int)at), page = g.table[(int64_t)n * g.max_pages + place];
    if (page >= 0 && page < g.n_pages)
      row[1] = static_cast<T*>(a.cache) + page * g.page_stride + row_in_page(g, (int)at, place) * g.row_stride;
  }
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (!row[w]) continue;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (64 * i + lane < CHUNKS) *reinterpret_cast<VecT*>(row[w] + (64 * i + lane) * E) = x[i];
    if (lane < DR / 2) {
      row[w][DC + ia] = from_f32<T>(pa);
      row[w][DC + ib] = from_f32<T>(pb);
    }
  }
}

// -- rotary -------------------------------------------------------------------------------

// A thread holds the angles of E / 2 (interleaved) or E (half) pairs of one token
// and walks the token's heads with them.
template <typename T, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a, int parts) {
  constexpr int E = 16 / sizeof(T), PAIRS = INTERLEAVED ? E / 2 : E;
  typedef T VecT __attribute__((ext_vector_type(E)));
  const int chunks = a.dim / (2 * PAIRS);  // threads a head takes
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = id / (chunks * parts);
  if (t >= a.t_total) return;
  const int rest = (int)(id - t * (chunks * parts)), part = rest / chunks, ch = rest - part * chunks;
  const double position = a.positions[t];
  float c[PAIRS], s[PAIRS];
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) turn_of(position, a.frequencies[ch * PAIRS + i], a.magnitude, c[i], s[i]);
  const T* x = static_cast<const T*>(a.x) + t * a.x_stride + ch * E;
  T* y = static_cast<T*>(a.y) + t * a.y_stride + ch * E;
  for (int h = part; h < a.n_heads; h += parts) {
    const T* xh = x + h * a.x_head;
    T* yh = y + h * a.y_head;
    if (INTERLEAVED) {
      const VecT u = *reinterpret_cast<const VecT*>(xh);
      VecT v;
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float p = (float)u[2 * i], q = (float)u[2 * i + 1];
        v[2 * i] = from_f32<T>(p * c[i] - q * s[i]);
        v[2 * i + 1] = from_f32<T>(q * c[i] + p * s[i]);
      }
      *reinterpret_cast<VecT*>(yh) = v;
    } else {
      const VecT u = *reinterpret_cast<const VecT*>(xh), w = *reinterpret_cast<const VecT*>(xh + a.dim / 2);
      VecT v, z;
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float p = (float)u[i], q = (float)w[i];
        v[i] = from_f32<T>(p * c[i] - q * s[i]);
        z[i] = from_f32<T>(q * c[i] + p * s[i]);
      }
      *reinterpret_cast<VecT*>(yh) = v;
      *reinterpret_cast<VecT*>(yh + a.dim / 2) = z;
    }
  }
}

template <typename T, int DC>
hipError_t append(const LatentAppendArgs& a, hipStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)a.pages.t_total + APPEND_TOKENS - 1) / APPEND_TOKENS);
  if (a.dr == 64) return enqueue(latent_append_kernel<T, DC, 64>, grid, 64 * APPEND_TOKENS, stream, a);
  return enqueue(latent_append_kernel<T, DC, 32>, grid, 64 * APPEND_TOKENS, stream, a);
}

template <typename T>
hipError_t rotary(const RotaryArgs& a, hipStream_t stream) {
  const int E = 16 / (int)sizeof(T), chunks = a.dim / (a.interleaved ? E : 2 * E);
  const int parts = a.n_heads < 8 ? a.n_heads : 8;  // threads that share a token's heads
  const unsigned grid = (unsigned)(((int64_t)a.t_total * chunks * parts + 255) / 256);
  if (a.interleaved) return enqueue(rotary_kernel<T, true>, grid, 256, stream, a, parts);
  return enqueue(rotary_kernel<T, false>, grid, 256, stream, a, parts);
}

}  // namespace

hipError_t launch_latent_append(const LatentAppendArgs& a, hipStream_t stream) {
  if (a.pages.t_total == 0) return hipSuccess;
  if (a.bf16) return a.dc == 512 ? append<bf16, 512>(a, stream) : append<bf16, 256>(a, stream);
  return a.dc == 512 ? append<float, 512>(a, stream) : append<float, 256>(a, stream);
}

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream) {
  if (a.t_total == 0) return hipSuccess;
  return a.bf16 ? rotary<bf16>(a, stream) : rotary<float>(a, stream);
}

}  // namespace kda
