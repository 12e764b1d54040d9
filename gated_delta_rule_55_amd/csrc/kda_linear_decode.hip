// kda_linear_decode.hip -- one token per (sequence, head) of linear attention
// with a decay per head, on a carried state that is updated in place
// (kda_linear_decode):
//     S <- exp(g) S + k v^T,   o = scale S^T q
//
// The step reads the state once and writes it once and is bound by that.  A
// workgroup owns CB value columns of one (sequence, head); a thread owns four
// of them in DK / RG consecutive rows, issues all its state loads before any
// arithmetic, and stores the updated values from registers.  o is the sum of
// q's rows times the new state, reduced over lanes and then through LDS.
//
// 64 sequences of 32 heads of 128 in fp32, 268 MB: 41 us (6.5 TB/s) back to back
// on one state, which then stays in the 256 MB cache in part, 52 us over three
// states in turn; 256 sequences, 1.07 GB: 210 us (5.1 TB/s, a copy's 4.75).
// CB is the whole row of DV columns, or 32 of them where there are fewer than
// 512 (sequence, head) pairs: one sequence of 32 heads is 128 workgroups
// then, and the 3.5 us that its launch takes anyway.
#include "kda_enqueue.h"
#include "kda_linear_launch.h"
#include "kda_linear_ops.h"

namespace kda {
namespace {

struct DecodeParams {
  void* state;
  const void *q, *k, *v;
  const float* g;
  void* o;
  int64_t qs, ks, vs, os;
  const int* slots;
  int H, rep, n_slots;
  float scale;
  bool decay_head;
};

template <typename T, typename TS, int DK, int DV, int CB>
__global__ __launch_bounds__(256) void linear_decode_kernel(DecodeParams P) {
  constexpr int NQ = CB / 4, RG = 256 / NQ, RPT = DK / RG, NC = DV / CB;
  static_assert(RG * RPT == DK && NC * CB == DV && NQ <= 64, "decode tiling");
  __shared__ float red[4][CB];
  const int cb = blockIdx.x % NC;
  const int nh = blockIdx.x / NC;
  const int n = nh / P.H, h = nh % P.H;
  int64_t slot = n;
  if (P.slots) {
    slot = P.slots[n];
    if (slot < 0 || slot >= P.n_slots) return;
  }
  const int tid = threadIdx.x, cq = tid % NQ, rg = tid / NQ;
  TS* S = static_cast<TS*>(P.state) + (slot * P.H + h) * (int64_t)(DK * DV) + (int64_t)rg * RPT * DV +
          cb * CB + 4 * cq;
  f32x4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) s[i] = load_state4(S + i * DV);
  const int hk = h / P.rep;
  const T* q = static_cast<const T*>(P.q) + n * P.qs + hk * DK + rg * RPT;
  const T* k = static_cast<const T*>(P.k) + n * P.ks + hk * DK + rg * RPT;
  float qr[RPT], kr[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    qr[i] = to_f32(q[i]);
    kr[i] = to_f32(k[i]);
  }
  const T* vp = static_cast<const T*>(P.v) + n * P.vs + h * DV + cb * CB + 4 * cq;
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = to_f32(vp[e]);
  const float g = P.decay_head ? P.g[h] : P.g[(int64_t)n * P.H + h];
  const float d = fast_exp2(g * kLog2e);
  f32x4 acc = zero4();
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    s[i] = s[i] * d + v * kr[i];
    acc += s[i] * qr[i];
  }
#pragma unroll
  for (int i = 0; i < RPT; ++i) store_state4(S + i * DV, s[i]);
#pragma unroll
  for (int off = NQ; off < 64; off <<= 1)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] += __shfl_xor(acc[e], off, 64);
  if ((tid & 63) < NQ) *reinterpret_cast<f32x4*>(&red[tid >> 6][4 * cq]) = acc;
  __syncthreads();
  if (tid < CB) {
    const float x = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
    static_cast<T*>(P.o)[n * P.os + h * DV + cb * CB + tid] = from_f32<T>(x * P.scale);
  }
}

template <typename T, typename TS, int DK, int DV>
hipError_t launch(const LinearDecodeArgs& a, const DecodeParams& p, hipStream_t stream) {
  const int64_t nh = (int64_t)a.n_seqs * a.n_heads;
  if (DV > 32 && nh < 512)
    return enqueue(linear_decode_kernel<T, TS, DK, DV, 32>, (unsigned)(nh * (DV / 32)), 256, stream, p);
  return enqueue(linear_decode_kernel<T, TS, DK, DV, DV>, (unsigned)nh, 256, stream, p);
}

template <typename T, typename TS>
hipError_t launch_dims(const LinearDecodeArgs& a, const DecodeParams& p, hipStream_t s) {
  switch (a.dk * 1000 + a.dv) {
    case 32032: return launch<T, TS, 32, 32>(a, p, s);
    case 32064: return launch<T, TS, 32, 64>(a, p, s);
    case 32128: return launch<T, TS, 32, 128>(a, p, s);
    case 64032: return launch<T, TS, 64, 32>(a, p, s);
    case 64064: return launch<T, TS, 64, 64>(a, p, s);
    case 64128: return launch<T, TS, 64, 128>(a, p, s);
    case 128032: return launch<T, TS, 128, 32>(a, p, s);
    case 128064: return launch<T, TS, 128, 64>(a, p, s);
    case 128128: return launch<T, TS, 128, 128>(a, p, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_linear_decode(const LinearDecodeArgs& a, hipStream_t stream) {
  DecodeParams p;
  p.state = a.state;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.g = a.g;
  p.o = a.o;
  p.qs = a.q_stride;
  p.ks = a.k_stride;
  p.vs = a.v_stride;
  p.os = a.o_stride;
  p.slots = a.slots;
  p.H = a.n_heads;
  p.rep = a.n_heads / a.kheads;
  p.n_slots = a.n_slots;
  p.scale = a.scale;
  p.decay_head = a.decay_head;
  if (!a.bf16) return launch_dims<float, float>(a, p, stream);
  return a.state_bf16 ? launch_dims<bf16, bf16>(a, p, stream) : launch_dims<bf16, float>(a, p, stream);
}

}  // namespace kda
