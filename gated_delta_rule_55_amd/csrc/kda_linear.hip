// kda_linear.hip -- linear attention with one decay per head over packed
// sequences (kda_linear_prefill).
//
// In chunks of 64 tokens (32 in fp32, and in bf16 where a launch of few tokens a
// sequence splits none), with G_i the sum of the log-decays of a chunk's tokens
// up to and with i, G the whole chunk's and S the state before it:
//     o_i = scale (exp(G_i) S^T q_i + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j)
//     S  <- exp(G) S + sum_j exp(G - G_j) k_j v_j^T
// Every factor is at most 1 when g <= 0.  The chunks of a sequence follow one
// another through S only, and S's decay over any run of tokens is one number,
// so a sequence longer than a segment of L tokens is split into P segments:
//     pass 1  every segment but the last: its own state from zero, and its decay
//     pass 2  S_in of each segment: S_in[p + 1] = decay_p S_in[p] + own_p
//     pass 3  every segment: its chunks from S_in, writing o; the last one hT
// A launch in which no sequence can be longer than L runs pass 3 alone.
//
// One workgroup walks a segment of one head with the state in registers: wave
// w owns value columns 32w .. 32w + 31, as dk / 32 D tiles (rows = key
// channels).  Q, K, V of a chunk lie in LDS; the next chunk's are loaded into
// registers while it is worked on.  All products are 32x32 MFMA steps:
//     scores^T = K Q^T     D tiles, decayed and masked, then through LDS as B
//     O^T      = S^T Q^T   S straight from its registers as A
//     O^T     += V^T P^T   V read transposed from LDS
//     S       += K^T V'    V' = exp(G - G_j) v_j
// V' in bf16 would cost the carried state half its digits, so it is split into
// three bf16 values (24 bits) and multiplied three times; q's copy of the
// state and P are rounded to bf16 once, as o will be.  (In two parts each they
// would bring o's error from 2.3e-3 to the 1.7e-3 of its own rounding, at 430 us
// against 396 for 32,768 tokens x 32 heads of 128.)
//
// What bounds it: the memory.  Of 32,768 tokens x 32 heads of 128 a kernel trace
// gives pass 1 141 us for the 0.57 GB that it moves, the rate of plain reading
// (4.0 TB/s), pass 2 13 us, and pass 3 265 us for 1.16 GB, at 4.4 TB/s near a
// copy's 4.75; the passes of an untraced call take 393 us together.  (With every
// product left out pass 3 took 239 us where it took 247 with them.)  What that
// leaves is k and v read twice: the segments' states are the price of 512
// workgroups for 32 chains.  Pass 3 in reverse order of segments, and the three
// passes over groups of heads, did not bring k and v back from the 256 MB cache;
// passes over blocks of tokens were not tried.
//
// Short calls are bound by the chain of their launches and chunks instead: one
// sequence of 32 heads of 128 takes 19 us for 256 tokens, 34 for 1,024, 46 for
// 2,048 and 79 for 4,096, which a copy would move in 3, 8, 15 and 29.
#include <type_traits>

#include "kda_enqueue.h"
#include "kda_linear_launch.h"
#include "kda_linear_ops.h"

namespace kda {
namespace {

constexpr int kGrain = 64;       // segments are multiples of this many tokens
constexpr float kMinG = -200.f;  // exp(-200) is 0 in fp32: -inf becomes a finite sum

struct LinearParams {
  const void *q, *k, *v;
  const float* g;
  void* o;
  int64_t qs, ks, vs, os;
  const void* h0;
  void* ht;
  const int32_t* cu;
  const int* slots;
  float* ws_state;  // [slot][H][dk][dv]
  float* ws_decay;  // [slot][H] natural log of a segment's decay
  int T, L;
  unsigned int lmul, lshift;  // x / L = (x / 64) * lmul >> lshift
  int N, H, rep, n_slots;
  float scale;
  bool state_bf16, decay_head;
};

struct Segment {
  int n, p, count;        // sequence, segment in it, its number of segments
  int begin, end;         // tokens
  int slot;               // workspace slot of segment 0
  int state;              // state slot of the sequence, negative: skip it
};

__device__ __forceinline__ int state_at(const LinearParams& P, int n) {
  if (!P.slots) return n;
  const int s = P.slots[n];
  return s < P.n_slots ? s : -1;
}

__device__ __forceinline__ int cu_at(const LinearParams& P, int n) {
  if (!P.cu) return n == 0 ? 0 : P.T;
  const int c = P.cu[n];
  return c < 0 ? 0 : c > P.T ? P.T : c;
}
__device__ __forceinline__ int div_l(const LinearParams& P, int x) {
  return (int)(((uint64_t)((unsigned int)x >> 6) * P.lmul) >> P.lshift);
}

// The segments of a sequence of `len` tokens: one (also of none), or equally
// long ones but for the last; `each` is their length.
__device__ __forceinline__ int count_segments(const LinearParams& P, int len, int& each) {
  each = P.L;
  if (len <= P.L) return 1;
  const unsigned int most = div_l(P, len - 1) + 1;
  each = (int)(((unsigned int)len + most - 1) / most + kGrain - 1) / kGrain * kGrain;
  return (int)(((unsigned int)len + each - 1) / (unsigned int)each);
}

__device__ __forceinline__ int len_of(int begin, int end) { return end > begin ? end - begin : 0; }

// Segment p of sequence n, which has `len` tokens from `begin`.
__device__ __forceinline__ Segment segment_of(const LinearParams& P, int n, int p, int begin, int len, int state) {
  Segment s;
  s.n = n;
  s.p = p;
  s.state = state;
  // sequences of two or more segments start in different L-token blocks, with
  // at least count - 1 blocks to the next such start: twice the block index
  // leaves room for count slots
  s.slot = 2 * div_l(P, begin);
  int each;
  s.count = count_segments(P, len, each);
  s.begin = begin + p * each;
  s.end = p + 1 < s.count ? s.begin + each : begin + len;
  return s;
}

// The last n with key(n) <= x for a key that does not fall, by one wave: each
// round narrows the range 64 times.
template <typename Key>
__device__ __forceinline__ int search(int n, int x, Key key) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int at = lo + lane * step;
    const bool in = lane * step < n && key(at) <= x;
    const int hits = __popcll(__ballot(in));
    const int skip = hits > 0 ? (hits - 1) * step : 0;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Segment `id` of the launch, by one wave: of all segments of all sequences
// (LAST), or of all but each sequence's last; at most T / L + N exist, and
// false comes back for ids without one.  Up to 64 sequences are counted by a
// lane each, and a scan numbers their segments without gaps.  Beyond that
// sequence n owns the T / L + N numbers from cu[n] / L + n on:
// cu[n + 1] / L - cu[n] / L + 1 of them, at least its ceil(len / L); those that
// it does not need are left out (counting 2,048 sequences of 32 tokens in every
// workgroup took 4.9 ms for what this does in 1.5).
template <bool LAST>
__device__ __forceinline__ bool find_segment(const LinearParams& P, int id, Segment& s) {
  if (P.N <= 64) {
    const int lane = threadIdx.x & 63;
    int mine = 0, each, begin = 0, len = 0, state = -1;
    if (lane < P.N) {
      begin = cu_at(P, lane);
      len = len_of(begin, cu_at(P, lane + 1));
      state = state_at(P, lane);
      mine = count_segments(P, len, each) - !LAST;
    }
    int sum = mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(sum, off, 64);
      if (lane >= off) sum += x;
    }
    const unsigned long long past = __ballot(sum > id);
    if (past == 0) return false;
    const int n = __builtin_ctzll(past);
    s = segment_of(P, n, id - __builtin_amdgcn_readlane(sum - mine, n), __builtin_amdgcn_readlane(begin, n),
                   __builtin_amdgcn_readlane(len, n), __builtin_amdgcn_readlane(state, n));
    return true;
  }
  // even numbers first: sequences of just L tokens leave out every other one,
  // which would leave every other XCD without work
  const int ids = div_l(P, P.T) + P.N, evens = (ids + 1) / 2;
  id = id < evens ? 2 * id : 2 * (id - evens) + 1;
  const int n = search(P.N, id, [&](int i) { return div_l(P, cu_at(P, i)) + i; });
  const int begin = cu_at(P, n);
  const int p = id - (div_l(P, begin) + n);
  s = segment_of(P, n, p, begin, len_of(begin, cu_at(P, n + 1)), state_at(P, n));
  return p >= 0 && p < s.count - !LAST;
}

// Which segment id and head group a workgroup takes.  Workgroups go round the
// 8 XCDs.  Where `share` groups of heads read one key head, these are 8 apart,
// so that they read q and k through the same L2; without that, neighbours in
// memory stay on different XCDs (the other way round cost 32,768 tokens x 32
// heads a quarter).
__device__ __forceinline__ void place(int groups, int share, int& id, int& group) {
  int i = blockIdx.x;
  if (share > 1) {
    const int r = i / 8 % share;
    i = (i / 8 / share * 8 + i % 8) * share + r;
  }
  id = i / groups;
  group = i % groups;
}
inline int64_t placed_blocks(int64_t ids, int groups, int share) {
  const int64_t n = ids * groups;
  return share > 1 ? (n / share + 7) / 8 * 8 * share : n;
}

// A wave's part of a state in memory, [DK][DV] at p of type TS, to or from its
// D tiles: register r of tile t is row 32t + 16 (r / 8) + 8 half + r % 8.
template <int DV, int KT, typename TS>
__device__ __forceinline__ void load_state(f32x16 (&S)[KT], const TS* p, int lane, int col0) {
  p += 8 * (lane >> 5) * DV + col0 + (lane & 31);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) S[t][r] = (float)p[(32 * t + 16 * (r >> 3) + (r & 7)) * DV];
}
template <int DV, int KT, typename TS>
__device__ __forceinline__ void store_state(const f32x16 (&S)[KT], TS* p, int lane, int col0) {
  p += 8 * (lane >> 5) * DV + col0 + (lane & 31);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) p[(32 * t + 16 * (r >> 3) + (r & 7)) * DV] = (TS)S[t][r];
}

// A chunk's rows of one of q, k, v on their way from memory to LDS, as 16-byte
// vectors.  Loads go through a buffer resource that ends with the chunk's last
// row, so rows past it read as zeros without a branch, and a thread's offsets
// are the same for every chunk.
template <typename T, int C, int D, int NT>
struct Rows {
  static constexpr int VE = 16 / sizeof(T);      // elements per vector
  static constexpr int VPR = D / VE;             // vectors per row
  static constexpr int RPP = NT / VPR;           // rows per step of the workgroup
  static constexpr int NV = C / RPP > 0 ? C / RPP : 1;
  static constexpr int S = D + 32 / sizeof(T);   // LDS row stride: 32 bytes of padding
  static_assert(NT % VPR == 0 && (C % RPP == 0 || RPP == 2 * C), "row tiling");
  uint4 r[NV];
  static __device__ __forceinline__ int offset(int tid, int64_t stride) {
    return ((tid / VPR) * (int)stride + (tid % VPR) * VE) * (int)sizeof(T);
  }
  // base: the chunk's first row; off: offset() of this thread
  __device__ __forceinline__ void load(const T* base, int off, int stride, int valid) {
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(const_cast<T*>(base), ((valid - 1) * stride + D) * (int)sizeof(T));
#pragma unroll
    for (int i = 0; i < NV; ++i)
      r[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, off + i * RPP * stride * (int)sizeof(T), 0, 0));
  }
  __device__ __forceinline__ void store(T* lds, int tid) const {
    if (RPP > C && tid / VPR >= C) return;
    T* p = lds + (tid / VPR) * S + (tid % VPR) * VE;
#pragma unroll
    for (int i = 0; i < NV; ++i) *reinterpret_cast<uint4*>(p + i * RPP * S) = r[i];
  }
};

// The decays of a chunk's tokens for one head, in powers of two.
template <int C>
struct Decays {
  alignas(16) float ghi[C], glo[C];  // G_i as a sum of two floats
  alignas(16) float eg[C], ed[C];    // exp(G_i), exp(G - G_i)
  float total;                       // exp(G)
};

// LDS of a workgroup: VW value columns (HG heads of VW / HG).
template <typename T, int C, int DK, int VW, int HG, bool OUT>
struct Smem {
  static constexpr int TILES = C / 32 * (C / 32 + 1) / 2;  // score tiles of a head
  alignas(16) T k[C * Rows<T, C, DK, 2 * VW>::S];
  alignas(16) T v[C * Rows<T, C, VW, 2 * VW>::S];
  alignas(16) T q[OUT ? C * Rows<T, C, DK, 2 * VW>::S : 8];
  alignas(16) T p[OUT ? HG * TILES * 2 * 64 * 8 : 8];  // score tiles as B operands
  Decays<C> d[2][HG];                                  // of this chunk and the next
};

// x of the lane that a data-parallel primitive's control names, 0 where there is
// none or the row of 16 lanes is not in ROWS.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const unsigned int lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned int)u, CTRL, ROWS, 0xf, true);
  const unsigned int hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive sums over the wave's lanes: within rows of 16 by shifts of 1, 2, 4
// and 8, then lane 15 of a row to the next one and lane 31 to the upper half.
// (Through LDS permutes the sums of two heads took longer than a score tile.)
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp<0x111, 0xf>(x);
  x += dpp<0x112, 0xf>(x);
  x += dpp<0x114, 0xf>(x);
  x += dpp<0x118, 0xf>(x);
  x += dpp<0x142, 0xa>(x);
  x += dpp<0x143, 0xc>(x);
  return x;
}

// One wave: the log-decay sums of a chunk and what is made of them.  Sums are
// fp64, and differences are taken from hi + lo pairs, so that a strong decay
// in the chunk does not cost the weaker ones after it their digits.  Returns G.
template <int C>
__device__ __forceinline__ double decay_sums(Decays<C>& d, float g, bool head, int valid, int lane) {
  g = g < kMinG ? kMinG : g;
  double G, all;
  if (head) {
    const int n = lane + 1 < valid ? lane + 1 : valid;
    G = (double)g * n;
    all = (double)g * valid;
  } else {
    G = wave_scan(lane < valid ? (double)g : 0.0);
    const uint64_t u = __builtin_bit_cast(uint64_t, G);
    const unsigned int lo = __builtin_amdgcn_readlane((int)(unsigned int)u, 63);
    const unsigned int hi = __builtin_amdgcn_readlane((int)(u >> 32), 63);
    all = __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  }
  constexpr double kL2E = 1.4426950408889634074;
  const double G2 = G * kL2E;
  const float hi = (float)G2;
  if (lane < C) {
    d.ghi[lane] = hi;
    d.glo[lane] = (float)(G2 - (double)hi);
    d.eg[lane] = fast_exp2(hi);
    d.ed[lane] = fast_exp2((float)((all - G) * kL2E));
  }
  if (lane == 0) d.total = fast_exp2((float)(all * kL2E));
  return all;
}

// Registers: __launch_bounds__ caps three output passes of bf16 where they spill a little
// (two heads of 64 a workgroup, dk 128: 2 of them in chunks of 64, 16 in chunks
// of 32; heads of 128 x 128 in chunks of 32: 3), for one more workgroup a CU.
// Workgroups of one or two waves, for heads of 32 and 64 that are not grouped,
// hold a whole dk x 32 state a wave and Q and K for themselves alone: with heads
// of 128 x 32 in bf16 a CU has room for three waves (8,192 tokens x 32 heads 98
// us; four heads to a key head, grouped, 59).
//
// Passes 1 (OUT = false) and 3 (OUT = true).  A workgroup walks one segment
// for HG heads that share a key head: VW value columns in all, 32 a wave.
// 64 sequences of 1,024 tokens, heads of 128 x 64, eight to a key head: 250 us
// with two heads a workgroup and the four workgroups of a key head on one XCD,
// 272 with them spread, 477 with one head a workgroup.
template <typename T, int C, int DK, int VW, int HG, bool OUT>
__global__ __launch_bounds__(2 * VW, sizeof(T) != 2 || VW != 128 || HG == 4 ? 1 : C == 32 ? 3 : 2)
void linear_kernel(LinearParams P) {
  constexpr int NW = VW / 32, NT = 64 * NW, KT = DK / 32, DV = VW / HG;
  constexpr int TT = C / 32;  // 32-token tiles of a chunk
  using RQ = Rows<T, C, DK, NT>;
  using RV = Rows<T, C, VW, NT>;
  using F = typename Frag<T>::type;
  using SM = Smem<T, C, DK, VW, HG, OUT>;
  __shared__ SM sm;

  const int groups = P.H / HG;
  int id, group;
  place(groups, P.rep / HG, id, group);
  const int hb = group * HG;  // first head
  Segment s;
  if (!find_segment<OUT>(P, id, s)) return;
  if (s.state < 0) return;

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int half = lane >> 5, col = lane & 31;
  const int hw = 32 * w / DV;  // this wave's head of the group
  const bool sbf = P.state_bf16;
  const int64_t sbase = ((int64_t)s.state * P.H + hb + hw) * (DK * DV);
  const int64_t wbase = ((int64_t)(s.slot + s.p) * P.H + hb + hw) * (DK * DV);
  const int col0 = 32 * w % DV;

  const int hk = hb / P.rep;
  const T* qb = OUT ? static_cast<const T*>(P.q) + s.begin * P.qs + hk * DK : nullptr;
  const T* kb = static_cast<const T*>(P.k) + s.begin * P.ks + hk * DK;
  const T* vb = static_cast<const T*>(P.v) + s.begin * P.vs + hb * DV;
  const int qo = OUT ? RQ::offset(tid, P.qs) : 0, ko = RQ::offset(tid, P.ks), vo = RV::offset(tid, P.vs);
  RQ rq, rk;
  RV rv;
  const int len = s.end - s.begin;
  auto valid_at = [&](int c0) { return len - c0 < C ? len - c0 : C; };
  auto fetch = [&](int c0) {
    const int valid = valid_at(c0);
    if (OUT) rq.load(qb + c0 * P.qs, qo, (int)P.qs, valid);
    rk.load(kb + c0 * P.ks, ko, (int)P.ks, valid);
    rv.load(vb + c0 * P.vs, vo, (int)P.vs, valid);
  };
  auto publish = [&]() {
    if (OUT) rq.store(sm.q, tid);
    rk.store(sm.k, tid);
    rv.store(sm.v, tid);
  };
  // the last wave, which has no score tile of its own when there are four,
  // holds the next chunk's log-decays and sums them a chunk ahead
  const bool gwave = w == NW - 1;
  float g[HG];
  double logsum[HG];
#pragma unroll
  for (int x = 0; x < HG; ++x) logsum[x] = 0.0;
  auto fetch_g = [&](int c0) {
#pragma unroll
    for (int x = 0; x < HG; ++x)
      g[x] = P.decay_head ? P.g[hb + x] : lane < valid_at(c0) ? P.g[(int64_t)(s.begin + c0 + lane) * P.H + hb + x] : 0.f;
  };
  auto sum_g = [&](int c0, int b) {
#pragma unroll
    for (int x = 0; x < HG; ++x) logsum[x] += decay_sums(sm.d[b][x], g[x], P.decay_head, valid_at(c0), lane);
  };

  // what is needed first is asked for first
  if (len > 0) {
    if (gwave) fetch_g(0);
    fetch(0);
  }
  f32x16 S[KT];
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) S[t][r] = 0.f;
  if (OUT) {
    if (s.count > 1) load_state<DV>(S, P.ws_state + wbase, lane, col0);
    else if (P.h0 && sbf) load_state<DV>(S, static_cast<const bf16*>(P.h0) + sbase, lane, col0);
    else if (P.h0) load_state<DV>(S, static_cast<const float*>(P.h0) + sbase, lane, col0);
  }
  if (len > 0) {
    if (gwave) {
      sum_g(0, 0);
      fetch_g(C);
    }
    publish();
  }
  __syncthreads();
  int buf = 0;
  for (int c0 = 0; c0 < len; c0 += C, buf ^= 1) {
    const bool more = c0 + C < len;
    if (more) {
      fetch(c0 + C);
      if (gwave) {
        sum_g(c0 + C, buf ^ 1);
        fetch_g(c0 + 2 * C);
      }
    }
    const Decays<C>& dw = sm.d[buf][hw];

    f32x16 O[TT];
    if (OUT) {
      // scores^T of tile (jt, it): rows = keys j, columns = queries i
#pragma unroll
      for (int tt = 0; tt < (SM::TILES + NW - 1) / NW; ++tt) {
        const int tile = w + tt * NW;
        if (tile >= SM::TILES) break;
        const int jt = tile >> 1, it = (tile + 1) >> 1;
        f32x16 a;
#pragma unroll
        for (int r = 0; r < 16; ++r) a[r] = 0.f;
        const T* krow = sm.k + (32 * jt + col) * RQ::S + 8 * half;
        const T* qrow = sm.q + (32 * it + col) * RQ::S + 8 * half;
#pragma unroll
        for (int x = 0; x < DK / 16; ++x) a = mma(load_frag8<T>(krow + 16 * x), load_frag8<T>(qrow + 16 * x), a);
        const int i = 32 * it + col;
#pragma unroll
        for (int hx = 0; hx < HG; ++hx) {
          const Decays<C>& d = sm.d[buf][hx];
          const float hi = d.ghi[i], lo = d.glo[i];
          f32x16 b;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int j = 32 * jt + 8 * x + 4 * half;
            const f32x4 jh = *reinterpret_cast<const f32x4*>(d.ghi + j);
            const f32x4 jl = *reinterpret_cast<const f32x4*>(d.glo + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float dec = fast_exp2((hi - jh[e]) + (lo - jl[e])) * P.scale;
              b[4 * x + e] = j + e <= i ? a[4 * x + e] * dec : 0.f;
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
            store_frag8(sm.p + (((hx * SM::TILES + tile) * 2 + x) * 64 + lane) * 8, frag_of_d<T>(b, x));
        }
      }
      // O^T = S^T Q^T, then the decay since the chunk's start and the scale
#pragma unroll
      for (int it = 0; it < TT; ++it)
#pragma unroll
        for (int r = 0; r < 16; ++r) O[it][r] = 0.f;
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const F sf = frag_of_d<T>(S[t], x);
#pragma unroll
          for (int it = 0; it < TT; ++it)
            O[it] = mma(sf, load_frag8<T>(sm.q + (32 * it + col) * RQ::S + 32 * t + 16 * x + 8 * half), O[it]);
        }
#pragma unroll
      for (int it = 0; it < TT; ++it) {
        const float e = dw.eg[32 * it + col] * P.scale;
#pragma unroll
        for (int r = 0; r < 16; ++r) O[it][r] *= e;
      }
    }

    // S = exp(G) S + K^T V'
    F vf[2 * TT];
    float poison = 0.f;  // NaN where a value is not finite
    const float total = dw.total;
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) S[t][r] *= total;
#pragma unroll
    for (int x = 0; x < 2 * TT; ++x) {
      vf[x] = frag_t<false>(sm.v + 16 * x * RV::S + 32 * w, RV::S, lane);
      poison = add_nonfinite(vf[x], poison);
      const f32x4 d0 = *reinterpret_cast<const f32x4*>(dw.ed + 16 * x + 4 * half);
      const f32x4 d1 = *reinterpret_cast<const f32x4*>(dw.ed + 16 * x + 8 + 4 * half);
      f32x8 vd;
#pragma unroll
      for (int e = 0; e < 8; ++e) vd[e] = to_f32(vf[x][e]) * (e < 4 ? d0[e & 3] : d1[e & 3]);
      if constexpr (sizeof(T) == 2) {
        bf16x8 vp[3];
        split3(vd, vp[0], vp[1], vp[2]);
        F kf[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) kf[t] = frag_t<true>(sm.k + 16 * x * RQ::S + 32 * t, RQ::S, lane);
        // the smallest part first; consecutive steps go to different tiles
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int t = 0; t < KT; ++t) S[t] = mma(kf[t], vp[part], S[t]);
      } else {
#pragma unroll
        for (int t = 0; t < KT; ++t)
          S[t] = mma(frag_t<true>(sm.k + 16 * x * RQ::S + 32 * t, RQ::S, lane), vd, S[t]);
      }
    }
    __syncthreads();  // the scores are written; this chunk's Q, K, V and decays are read
    if (more) publish();

    if (OUT) {
      const bool bad = __any(poison != 0.f);
      if (bad) {  // a masked score of 0 would turn these into NaN: added below
#pragma unroll
        for (int x = 0; x < 2 * TT; ++x)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!finite1(to_f32(vf[x][e]))) vf[x][e] = from_f32<T>(0.f);
      }
      const T* pw = sm.p + hw * SM::TILES * 2 * 64 * 8;
#pragma unroll
      for (int tile = 0; tile < SM::TILES; ++tile) {
        const int jt = tile >> 1, it = (tile + 1) >> 1;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          O[it] = mma(vf[2 * jt + x], load_frag8<T>(pw + ((tile * 2 + x) * 64 + lane) * 8), O[it]);
      }
      const int valid = valid_at(c0);
      if (bad) {
#pragma unroll 1
        for (int j = 0; j < valid; ++j) {
          const T* vrow = vb + (int64_t)(c0 + j) * P.vs + 32 * w;
          const int jt = j >> 5, x = (j >> 4) & 1, jj = j & 15;
          const int e = (jj & 3) + 4 * (jj >> 3), jlane = 32 * ((jj >> 2) & 1) + col;
          float pj[TT];  // P[i][j] of this lane's two queries
#pragma unroll
          for (int it = 0; it < TT; ++it)
            pj[it] = jt <= it ? to_f32(pw[(((jt + it) * 2 + x) * 64 + jlane) * 8 + e]) : 0.f;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float x1 = to_f32(vrow[d_row(r, half)]);
            if (!finite1(x1)) {
#pragma unroll
              for (int it = 0; it < TT; ++it)
                if (32 * it + col >= j) O[it][r] += pj[it] * x1;
            }
          }
        }
      }
      // lane: token 32 it + col, value columns 8 (r / 4) + 4 half + r % 4
#pragma unroll
      for (int it = 0; it < TT; ++it) {
        const int i = 32 * it + col;
        T* op = static_cast<T*>(P.o) + (int64_t)(s.begin + c0 + i) * P.os + hb * DV + 32 * w;
        if constexpr (sizeof(T) == 2) {
          // the halves trade register groups, so that each holds 8 columns in a row
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            typedef bf16 b2 __attribute__((ext_vector_type(2)));
            unsigned int lo[2], hi[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              lo[e] = __builtin_bit_cast(unsigned int, b2{(bf16)O[it][8 * y + 2 * e], (bf16)O[it][8 * y + 2 * e + 1]});
              hi[e] = __builtin_bit_cast(unsigned int, b2{(bf16)O[it][8 * y + 4 + 2 * e], (bf16)O[it][8 * y + 5 + 2 * e]});
            }
            const auto s0 = __builtin_amdgcn_permlane32_swap(lo[0], hi[0], false, false);
            const auto s1 = __builtin_amdgcn_permlane32_swap(lo[1], hi[1], false, false);
            if (i < valid)
              *reinterpret_cast<uint4*>(op + 16 * y + 8 * half) = uint4{s0[0], s1[0], s0[1], s1[1]};
          }
        } else {
          if (i < valid) {
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<f32x4*>(op + 8 * y + 4 * half) =
                  f32x4{O[it][4 * y], O[it][4 * y + 1], O[it][4 * y + 2], O[it][4 * y + 3]};
          }
        }
      }
    }
    __syncthreads();  // the next chunk is in LDS
  }

  if (OUT) {
    if (P.ht && s.p + 1 >= s.count) {
      if (sbf) store_state<DV>(S, static_cast<bf16*>(P.ht) + sbase, lane, col0);
      else store_state<DV>(S, static_cast<float*>(P.ht) + sbase, lane, col0);
    }
  } else {
    store_state<DV>(S, P.ws_state + wbase, lane, col0);
    if (gwave && lane == 0) {
#pragma unroll
      for (int x = 0; x < HG; ++x) P.ws_decay[(int64_t)(s.slot + s.p) * P.H + hb + x] = (float)logsum[x];
    }
  }
}

// Pass 2: the state each segment of a split sequence starts from, in place of
// the segments' own states.  A thread walks X vectors of four elements through
// the segments, up to 16 / X segments loaded at a time; bound by the workspace's
// traffic (32,768 tokens x 32 heads: 12 us), two vectors a thread keeping the
// workgroups few, or by the walk where there are few of them: one vector then.
// Workgroups go by sequence or, where there are more sequences than segment
// lengths in the batch, by the multiples of L: a sequence of two or more
// segments holds one behind its first token, and its first such takes it.
template <int X>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearParams P, int elems, int parts, bool marks) {
  const int e = (blockIdx.x % parts * blockDim.x + threadIdx.x) * 4 * X;
  const int nh = blockIdx.x / parts;
  const int h = nh % P.H;
  int n = nh / P.H;
  const int block = n + 1;
  if (marks) n = search(P.N, block * P.L - 1, [&](int i) { return cu_at(P, i); });
  const int begin = cu_at(P, n);
  const Segment s = segment_of(P, n, 0, begin, len_of(begin, cu_at(P, n + 1)), state_at(P, n));
  if (s.count < 2 || (marks && s.slot / 2 + 1 != block) || e >= elems || s.state < 0) return;
  f32x4 S[X];
#pragma unroll
  for (int x = 0; x < X; ++x) S[x] = zero4();
  if (P.h0) {
    const int64_t b = ((int64_t)s.state * P.H + h) * elems + e;
#pragma unroll
    for (int x = 0; x < X; ++x)
      S[x] = P.state_bf16 ? load_state4(static_cast<const bf16*>(P.h0) + b + 4 * x)
                          : load_state4(static_cast<const float*>(P.h0) + b + 4 * x);
  }
  const int64_t step = (int64_t)P.H * elems;
  float* p = P.ws_state + ((int64_t)s.slot * P.H + h) * elems + e;
  const float* d = P.ws_decay + (int64_t)s.slot * P.H + h;
  const int own = s.count - 1;  // segments with a state of their own
  auto walk = [&](auto count) {
    constexpr int K = decltype(count)::value;
    f32x4 own_s[K][X];
    float dec[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
      for (int x = 0; x < X; ++x) own_s[j][x] = *reinterpret_cast<const f32x4*>(p + j * step + 4 * x);
      dec[j] = d[j * P.H];
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const float f = fast_exp2(dec[j] * kLog2e);
#pragma unroll
      for (int x = 0; x < X; ++x) {
        *reinterpret_cast<f32x4*>(p + j * step + 4 * x) = S[x];
        S[x] = S[x] * f + own_s[j][x];
      }
    }
    p += K * step;
    d += K * P.H;
  };
  // the loads of up to B segments are in flight together (63 segments of 16 heads
  // of 64 x 64: 9.5 us, with 4 of them 10.7)
  constexpr int B = 16 / X;
  for (int i = 0; i < own / B; ++i) walk(std::integral_constant<int, B>{});
  if (X == 1 && (own & 8)) walk(std::integral_constant<int, 8>{});
  if (own & 4) walk(std::integral_constant<int, 4>{});
  if (own & 2) walk(std::integral_constant<int, 2>{});
  if (own & 1) walk(std::integral_constant<int, 1>{});
#pragma unroll
  for (int x = 0; x < X; ++x) *reinterpret_cast<f32x4*>(p + 4 * x) = S[x];
}

// Tokens per chunk.  fp32 takes twice the LDS and registers a token: with 64 its
// workgroups leave a SIMD one wave, of heads of 128 x 32 even a CU (8,192 tokens
// x 32 heads: 554 us against 182).
template <typename T>
constexpr int kChunk = sizeof(T) == 2 ? 64 : 32;

template <typename T, int DK, int DV, int HG>
hipError_t launch(const LinearParams& p, bool split, hipStream_t stream) {
  const int64_t blocks = placed_blocks(linear_segments(p.T, p.N, p.L), p.H / HG, p.rep / HG);
  constexpr int VW = DV * HG;
  if (split) {
    hipError_t e = enqueue(linear_kernel<T, kChunk<T>, DK, VW, HG, false>, (unsigned)blocks, 2 * VW, stream, p);
    if (e != hipSuccess) return e;
    constexpr int parts = DK * DV / 1024, parts2 = (parts + 1) / 2;
    const bool marks = p.T / p.L < p.N;
    const int64_t most = (int64_t)(marks ? p.T / p.L : p.N) * p.H;
    // workgroups of a wave where those of four would leave CUs without one (63
    // segments of 16 heads of 64 x 64: 9.5 us against 11.6)
    if (most * parts <= 128)
      e = enqueue(linear_join_kernel<1>, (unsigned)(most * parts * 4), 64, stream, p, DK * DV, parts * 4, marks);
    else if (most * parts <= 512)
      e = enqueue(linear_join_kernel<1>, (unsigned)(most * parts), 256, stream, p, DK * DV, parts, marks);
    else
      e = enqueue(linear_join_kernel<2>, (unsigned)(most * parts2), 256, stream, p, DK * DV, parts2, marks);
    if (e != hipSuccess) return e;
  }
  // Sequences of few tokens in bf16 are mostly loads and stores of states: chunks
  // of 32 leave room for three workgroups a CU (24 sequences of 851 tokens in all,
  // 32 heads of 128: 20 us against 24).  Longer ones lose a little by it (64 x
  // 1,024 tokens: 267 us against 256).  That is asked of the batch's average, and
  // only where no sequence can be split: a batch of more tokens than a segment
  // (1,024 from 256 sequences x heads on) runs all three passes in chunks of 64,
  // however short its sequences are (64 x 20 tokens: 54 us, a copy's time 37).
  if constexpr (sizeof(T) == 2) {
    if (!split && p.T <= 64 * (int64_t)p.N)
      return enqueue(linear_kernel<T, 32, DK, VW, HG, true>, (unsigned)blocks, 2 * VW, stream, p);
  }
  return enqueue(linear_kernel<T, kChunk<T>, DK, VW, HG, true>, (unsigned)blocks, 2 * VW, stream, p);
}

// Heads narrower than 128 that share a key head are taken together, four waves
// to a workgroup: q, k and the scores' products are read and made once for them.
template <typename T, int DK>
hipError_t launch_dk(const LinearParams& p, int dv, bool split, hipStream_t s) {
  switch (dv) {
    case 32: return p.rep % 4 == 0 ? launch<T, DK, 32, 4>(p, split, s) : launch<T, DK, 32, 1>(p, split, s);
    case 64: return p.rep % 2 == 0 ? launch<T, DK, 64, 2>(p, split, s) : launch<T, DK, 64, 1>(p, split, s);
    case 128: return launch<T, DK, 128, 1>(p, split, s);
    default: return hipErrorInvalidValue;
  }
}

template <typename T>
hipError_t launch_dims(const LinearParams& p, int dk, int dv, bool split, hipStream_t s) {
  switch (dk) {
    case 32: return launch_dk<T, 32>(p, dv, split, s);
    case 64: return launch_dk<T, 64>(p, dv, split, s);
    case 128: return launch_dk<T, 128>(p, dv, split, s);
    default: return hipErrorInvalidValue;
  }
}

size_t decay_bytes(int64_t slots, int H) { return ((size_t)slots * H * 4 + 255) / 256 * 256; }
int64_t ws_slots(int64_t T, int64_t L) { return 2 * (T / L) + 1; }

}  // namespace

int64_t linear_segment(int64_t t_total, int n_seqs, int n_heads, int dv, bool bf16) {
  // about eight waves, of 32 value columns each, for each of the 256 CUs (one
  // sequence of 32,768 tokens x 32 heads: 400 us, with twelve 455, sixteen 424);
  // for several sequences, whose segments are not equally long, twelve (eight of
  // 33,001 tokens in all: 395 us, with eight or sixteen 455 to 460).  Steps of
  // that size come from how segments fill the last round of 512 workgroups; other
  // lengths may do better with another number.
  const int64_t waves = 256 * (n_seqs == 1 ? 8 : 12);
  const int64_t want = (t_total * n_heads * (dv / 32) + waves - 1) / waves;
  int64_t seg = (want + kGrain - 1) / kGrain * kGrain;
  // segments of one or two chunks leave most of the time to launches, states and
  // their join: half as many then (2,048 tokens x 32 heads: 51 us -> 48; 4,096,
  // whose segments have four, 71 -> 73)
  if (bf16 && seg <= 128) seg = (2 * want + kGrain - 1) / kGrain * kGrain;
  // below that a split costs two launches more: taken for short sequences only
  // when they alone leave CUs idle (512 tokens x 32 heads in bf16: 31 us against
  // 32 in one segment, 1,024: 36 against 59), and not for 256 tokens (26 against
  // 19; in fp32, whose products take longer, 24 against 42 for 16 heads of 64)
  const int64_t least = (int64_t)n_seqs * n_heads >= 256 ? 1024 : !bf16 ? 64 : t_total <= 256 ? 256 : 128;
  return seg < least ? least : seg;
}

size_t linear_workspace_bytes(const LinearPrefillArgs& a) {
  const int64_t L = linear_segment(a.t_total, a.n_seqs, a.n_heads, a.dv, a.bf16);
  if (a.t_total <= L) return 0;
  const int64_t slots = ws_slots(a.t_total, L);
  return decay_bytes(slots, a.n_heads) + (size_t)slots * a.n_heads * a.dk * a.dv * 4;
}

hipError_t launch_linear_prefill(const LinearPrefillArgs& a, void* workspace, hipStream_t stream) {
  LinearParams p;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.g = a.g;
  p.o = a.o;
  p.qs = a.q_stride;
  p.ks = a.k_stride;
  p.vs = a.v_stride;
  p.os = a.o_stride;
  p.h0 = a.h0;
  p.ht = a.ht;
  p.cu = a.cu_seqlens;
  p.slots = a.slots;
  p.T = (int)a.t_total;
  p.L = (int)linear_segment(a.t_total, a.n_seqs, a.n_heads, a.dv, a.bf16);
  // x / 64 < 2^25 and L / 64 <= 2^k: exact with lmul = ceil(2^(25 + k) / (L / 64))
  const uint64_t l = (uint64_t)p.L / 64;
  unsigned int k = 0;
  while (((uint64_t)1 << k) < l) ++k;
  p.lshift = 25 + k;
  p.lmul = (unsigned int)((((uint64_t)1 << p.lshift) + l - 1) / l);
  p.N = a.n_seqs;
  p.H = a.n_heads;
  p.rep = a.n_heads / a.kheads;
  p.n_slots = a.n_slots;
  p.scale = a.scale;
  p.state_bf16 = a.state_bf16;
  p.decay_head = a.decay_head;
  const bool split = a.t_total > p.L;
  p.ws_decay = static_cast<float*>(workspace);
  p.ws_state = split ? reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) +
                                                decay_bytes(ws_slots(p.T, p.L), p.H))
                     : nullptr;
  return a.bf16 ? launch_dims<bf16>(p, a.dk, a.dv, split, stream)
                : launch_dims<float>(p, a.dk, a.dv, split, stream);
}

}  // namespace kda
