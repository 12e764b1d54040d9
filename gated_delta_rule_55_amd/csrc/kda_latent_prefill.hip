// kda_latent_prefill.hip -- expanded latent attention over packed prompts
// (kda_latent_prefill): o_i = sum_j p_ij v_j with p_ij the softmax over the keys
// j <= i + Lk - Lq of scale (q_i[:dn] . k_j + q_i[dn:] . k_pe_j).
//
// A workgroup takes 128 queries of one head, 32 to a wave, and walks the keys in
// tiles of 64 that all four waves read from LDS: scores transposed (S^T = K Q^T,
// a query per lane), the running maximum m and sum l of the softmax in fp32, and
// O^T += V^T P^T with the weights straight from the score registers.  O is scaled
// by 2^(m_old - m_new) where a maximum grew.
//
// Every key is read from LDS by four waves and every tile by all workgroups of its
// head, so it is the matrix cores, the vector unit (exponentials, maxima, sums) and
// LDS that bound it, not the memory.  Two tiles, one worked on while the other is
// fetched straight into LDS, take 80 KB in bf16: two workgroups a CU, so that one's
// softmax runs beside the other's products; fp32 takes 160 KB, one.  32,768 tokens, 32
// heads of 128 + 64, bf16: 10.8 to 11.2 ms on different cards, 0.98 to 1.02 PFLOP/s where a large
// matrix product reaches 1.18; matrix cores busy for 52 % of the cycles (the clock is at 1.8 GHz
// under this load), LDS for 43 %.  Waves of a block that have no query work along, on rows
// that are not stored: a sequence of up to 32 queries costs the products of 128.
//
// In bf16 the weights are rounded before they meet the values (2^-8 of a weight at most), since the
// matrix cores take operands of one type and fp32's run at an eighth of the rate; a second
// product for the rest of each weight is 40 % more of them and does not fit the registers (15.4 ms
// for 10.9).  Their sum is taken before that.  Against float64 the outputs' error grows from that
// of their own rounding, 1.6e-3 of their norm, to 1.9e-3.
#include <algorithm>

#include "kda_enqueue.h"
#include "kda_latent_launch.h"
#include "kda_latent_ops.h"

namespace kda {
namespace {

constexpr int QB = kLatentQueryBlock, KB = 64, THREADS = 256;

// Where the blocks are too few for the GPU, a block's tiles go to up to `parts`
// workgroups in equal shares; each leaves its unnormalised sums, its maxima and its
// sums of weights in the workspace, and latent_prefill_join_kernel adds them up.
// Measured, alone and shared (16 heads of 128 + 64, us): bf16, 256 queries on 8,192 keys
// 198 and 50, 1,000 on 16,000 376 and 193, 128 on 1,024 33 and 20, 512 on 512 22 and 23;
// fp32, 64 on 4,096 692 and 63.
constexpr int PART_TILES = 2;  // of a share, if it is not all (128 queries on 1,024 keys: 1 24 us, 2 and 4 20)
struct Parts {
  int parts;
  float* sums;    // [parts][q_total][H][dv]
  float2* stats;  // [parts][q_total][H]: maximum (of scores), sum of weights
  __host__ __device__ __forceinline__ int share(int tiles) const {
    const int by = min(parts, max(tiles / PART_TILES, 1));
    return (tiles + by - 1) / by;
  }
};

int parts_of(const LatentPrefillArgs& a) {
  // workgroups that run at a time: tiles leave room for two per CU in bf16, one in fp32
  const int64_t slots = a.bf16 ? 512 : 256, blocks = latent_query_blocks(a.q_total, a.n_seqs) * a.n_heads;
  return (int)std::max(std::min(slots / blocks, ((int64_t)a.k_total + KB - 1) / KB / PART_TILES), (int64_t)1);
}

// Keys, positional parts and values of a tile, each in whole column blocks.
template <typename T, int DN, int DR, int DV>
struct Tile {
  static constexpr int ES = sizeof(T);
  static constexpr int kn = DN * ES / 128, kp = (DR * ES + 127) / 128, kv = DV * ES / 128;
  static constexpr int pe = kn * KB * 128, v = pe + kp * KB * 128, bytes = v + kv * KB * 128;
};

template <typename T, int DN, int DR, int DV>
struct Prefill {
  using L = Tile<T, DN, DR, DV>;
  using F = typename Frag<T>::type;
  static constexpr int KS = (DN + DR) / 16, NV = DV / 32;

  F q[KS];
  f32x16 o[NV];
  float m, l;
  bool special;
  RowFrags<T, KB, 16> key_frags;
  ColFrags<T, KB> value_frags;

  __device__ __forceinline__ explicit Prefill(int lane)
      : m(-__builtin_inff()), l(0.f), special(false), key_frags(lane & 31, lane >> 5), value_frags(0, lane) {
#pragma unroll
    for (int d = 0; d < NV; ++d) o[d] = zero16();
  }

  // One tile's keys from position `key0` on, of which this lane's query sees those
  // up to `last`.  MASKED: some query of the wave does not see all of them; where such a
  // tile holds a value that is not finite, `special` is set and SAFE does the block again.
  template <bool MASKED, bool SAFE>
  __device__ __forceinline__ void step(const char* lds, int key0, int last, float c, int lane) {
    const int h = lane >> 5;
    f32x16 s[2] = {zero16(), zero16()};
    pipelined<F, 2 * KS, 4>(
        [&](int i) {
          const int k = i / 2, t = i % 2;
          return 16 * k < DN ? key_frags.load(lds, k, 32 * t) : key_frags.load(lds + L::pe, k - DN / 16, 32 * t);
        },
        [&](int i, F key) { s[i % 2] = mma16(key, q[i / 2], s[i % 2]); });
    if (MASKED) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (key0 + 32 * t + row_of(h, i) > last) s[t][i] = -__builtin_inff();
    }
    float top = m;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
    top = max_halves(top);
    // (a maximum's product with c is rounded the same way each time it is formed)
    const float base = top == -__builtin_inff() ? 0.f : __fmul_rn(top, c);
    const float alpha = fast_exp2(__fmul_rn(m, c) - base);
    m = top;
    float sum = 0.f;
    F p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float x = fast_exp2(s[t][i] * c - base);
        sum += x;
        p[2 * t + (i >> 3)][i & 7] = from_f32<T>(x);  // bf16: one rounding, 2^-8 (see the top)
      }
    l = l * alpha + sum;
    if (__builtin_expect(__any(alpha != 1.f), 0)) {
#pragma unroll
      for (int d = 0; d < NV; ++d) o[d] *= alpha;
    }
    const char* values = lds + L::v;
    if (MASKED && SAFE) {
      values_special(values, p, key0, last, lane);
      return;
    }
    if (MASKED) special |= not_finite(values, lane);
    pipelined<F, 4 * NV, 2>([&](int i) { return value_frags.load(values, 16 * (i % 4), i / 4); },
                            [&](int i, F value) { o[i / 4] = mma16(value, p[i % 4], o[i / 4]); });
  }

  // Whether a tile holds a value that is not finite.
  static __device__ __forceinline__ bool not_finite(const char* values, int lane) {
    bool any = false;
#pragma unroll
    for (int b = 0; b < L::kv * KB * 128 / 1024; ++b) {
      const uint4 x = *reinterpret_cast<const uint4*>(values + b * 1024 + lane * 16);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 2)
          any |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
        else
          any |= (w[i] & 0x7f800000u) == 0x7f800000u;
      }
    }
    return any;
  }
  __device__ __forceinline__ void values_special(const char* values, const F (&p)[4], int key0, int last, int lane) {
    const int h = lane >> 5;
#pragma unroll
    for (int d = 0; d < NV; ++d) {
      f32x16 kinds = zero16();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        F v = value_frags.load(values, 16 * k, d), kind, sees;
        split_special(v, kind);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          sees[e] = from_f32<T>(key0 + 16 * k + 8 * (e >> 2) + 4 * h + (e & 3) <= last ? 1.f : 0.f);
        o[d] = mma16(v, p[k], o[d]);
        kinds = mma16(kind, sees, kinds);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] = add_special(o[d][i], kinds[i]);
    }
  }
};

// Queries first .. first + QB - 1 of a sequence, of one head: its queries begin at q0, its
// keys at k0.
template <typename T, int DN, int DR, int DV, bool SAFE>
__device__ __forceinline__ bool prefill_block(const LatentPrefillArgs& a, const Parts& split, char* even, char* odd,
                                              int head, int first, int q0, int queries, int k0, int keys, int part) {
  using P = Prefill<T, DN, DR, DV>;
  using L = Tile<T, DN, DR, DV>;
  constexpr int ES = sizeof(T);
  const int lane = threadIdx.x & 63, wave = wave_index(), h = lane >> 5;
  const int mine = first + 32 * wave + (lane & 31);
  const int last = mine + (keys - queries);                     // the last key this lane's query sees
  const int wave_last = first + 32 * wave + (keys - queries);   // the last one that all of the wave's see
  // keys that the workgroup's last query sees
  const int end = min(first + QB, queries) + (keys - queries);

  P s(lane);
  {
    const char* row = static_cast<const char*>(a.q) +
                      ((int64_t)(q0 + min(mine, queries - 1)) * a.q_stride + (int64_t)head * (DN + DR) + 8 * h) * ES;
#pragma unroll
    for (int k = 0; k < P::KS; ++k) s.q[k] = load_frag8<T>(reinterpret_cast<const T*>(row + 16 * k * ES));
  }

  // The next tile is fetched while one is worked on.  A wave fetches 16 rows of it,
  // eight lanes to 128 bytes of a row, the chunks exchanged as tile_at has them.
  const float c = a.scale * kLog2e;
  const int r0 = 16 * wave + (lane >> 3), chunk = ((lane & 7) ^ row_swap(lane >> 3)) * 16;
  const int k_row = (int)a.k_stride * ES, p_row = (int)a.pe_stride * ES, v_row = (int)a.v_stride * ES;
  const char* kt = static_cast<const char*>(a.k) + (k0 * a.k_stride + head * a.k_head) * ES;
  const char* pt = static_cast<const char*>(a.pe) + k0 * a.pe_stride * ES;
  const char* vt = static_cast<const char*>(a.v) + (k0 * a.v_stride + head * a.v_head) * ES;
  auto fetch = [&](int t, char* tile) {
    // rows past the sequence, which are another's or nobody's, are 0
    const int rows = min(keys - t * KB, KB) - 1;
    const auto kr = make_rsrc(const_cast<char*>(kt + (int64_t)t * KB * k_row), rows * k_row + DN * ES);
    const auto pr = make_rsrc(const_cast<char*>(pt + (int64_t)t * KB * p_row), rows * p_row + DR * ES);
    const auto vr = make_rsrc(const_cast<char*>(vt + (int64_t)t * KB * v_row), rows * v_row + DV * ES);
    char* at = tile + 16 * wave * 128;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = r0 + 8 * r;
#pragma unroll
      for (int x = 0; x < L::kn; ++x) fetch16(kr, row * k_row + chunk, 128 * x, at + (x * KB + 8 * r) * 128);
#pragma unroll
      for (int x = 0; x < L::kp; ++x) {
        // a positional row narrower than a column block: the other lanes' chunks are not read
        const bool in = 128 * x + chunk < DR * ES;
        fetch16(pr, in ? row * p_row + chunk : kBufferOff, 128 * x, at + L::pe + (x * KB + 8 * r) * 128);
      }
#pragma unroll
      for (int x = 0; x < L::kv; ++x) fetch16(vr, row * v_row + chunk, 128 * x, at + L::v + (x * KB + 8 * r) * 128);
    }
  };
  auto work = [&](int t, const char* tile) {
    if (__builtin_expect(t * KB + KB - 1 <= wave_last, 1))
      s.template step<false, SAFE>(tile, t * KB, last, c, lane);
    else if (t * KB <= wave_last + 31)
      s.template step<true, SAFE>(tile, t * KB, last, c, lane);
  };
  const int all = end > 0 ? (end + KB - 1) / KB : 0, share = split.share(all);
  const int begin = part * share, tiles = min(begin + share, all);
  if (part > 0 && begin >= all) return true;
  if (begin < tiles) fetch(begin, even);
  for (int t = begin; t < tiles; t += 2) {
    fetched();
    if (t + 1 < tiles) fetch(t + 1, odd);
    work(t, even);
    if (t + 1 == tiles) break;
    fetched();
    if (t + 2 < tiles) fetch(t + 2, even);
    work(t + 1, odd);
  }

  if (!SAFE) {  // (the flags go where the tiles were: there is no room beside them)
    int* flags = reinterpret_cast<int*>(even);
    const bool special = __any(s.special);
    __syncthreads();
    flags[wave] = special;
    __syncthreads();
    const bool any = __any(flags[lane & 3]);
    __syncthreads();
    if (any) return false;
  }
  const float sum = s.l + other_half(s.l);
  if (share < all) {
    const int64_t place = ((int64_t)part * a.q_total + q0 + first) * a.n_heads + head;
    const auto sums = make_rsrc(split.sums + place * DV, INT32_MAX), stats = make_rsrc(split.stats + place, INT32_MAX);
    const int row = (mine - first) * a.n_heads;  // (few heads: below 2^16)
#pragma unroll
    for (int d = 0; d < P::NV; ++d)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 y = {s.o[d][4 * g], s.o[d][4 * g + 1], s.o[d][4 * g + 2], s.o[d][4 * g + 3]};
        store4(y, sums, mine < queries ? (row * DV + 32 * d + 8 * g + 4 * h) * 4 : kBufferOff);
      }
    const u32x2 st = {__float_as_uint(s.m), __float_as_uint(sum)};
    __builtin_amdgcn_raw_buffer_store_b64(st, stats, mine < queries && h == 0 ? row * 8 : kBufferOff, 0, 0);
    end_of_variant<SAFE>();
    return true;
  }
  const float inv = last >= 0 ? __builtin_amdgcn_rcpf(sum) : 0.f;  // no key: O is 0
  const auto out = make_rsrc(static_cast<char*>(a.o) + ((int64_t)(q0 + first) * a.o_stride + head * DV) * ES, INT32_MAX);
  const int at = (int)((mine - first) * a.o_stride + 4 * h) * ES;
#pragma unroll
  for (int d = 0; d < P::NV; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      typename Vec4<T>::type y;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(s.o[d][4 * g + e] * inv);
      store4(y, out, mine < queries ? at + (32 * d + 8 * g) * ES : kBufferOff);
    }
  end_of_variant<SAFE>();
  return true;
}

template <typename T, int DN, int DR, int DV>
__global__ __launch_bounds__(THREADS, sizeof(T) == 2 ? 2 : 1) void latent_prefill_kernel(LatentPrefillArgs a, Parts split,
                                                                                           int blocks, int classes) {
  using L = Tile<T, DN, DR, DV>;
  __shared__ __attribute__((aligned(128))) char even[L::bytes], odd[L::bytes];
  // Workgroups go round the 8 XCDs; those of one XCD take the heads of one class, a
  // head after the other, so that the workgroups that run together there read the
  // same keys through its L2.  Late queries, which see most keys, go first.
  const int xcd = blockIdx.x & 7, per = 8 / classes, part = (blockIdx.x >> 3) % split.parts;
  const int i = (blockIdx.x >> 3) / split.parts;
  const int nb = (blocks + per - 1) / per;
  const int head = xcd / per + classes * (i / nb);
  const int back = xcd % per + per * (i % nb);
  if (back >= blocks) return;
  const int64_t b = blocks - 1 - back;
  const int n = find_sequence<QB>(a.cu, a.n_seqs, a.q_total, 1, b);
  const int q0 = a.cu ? seq_start(a.cu, n, a.q_total) : 0, q1 = a.cu ? seq_start(a.cu, n + 1, a.q_total) : a.q_total;
  const int64_t block = b - first_block<QB>(q0, 1, n);
  if (block < 0 || block * QB >= q1 - q0) return;
  const int32_t* cu_k = a.cu_k ? a.cu_k : a.cu;
  const int k0 = cu_k ? seq_start(cu_k, n, a.k_total) : 0, k1 = cu_k ? seq_start(cu_k, n + 1, a.k_total) : a.k_total;
  const int first = (int)block * QB, keys = max(k1 - k0, 0);
  if (!prefill_block<T, DN, DR, DV, false>(a, split, even, odd, head, first, q0, q1 - q0, k0, keys, part))
    prefill_block<T, DN, DR, DV, true>(a, split, even, odd, head, first, q0, q1 - q0, k0, keys, part);
}

// The rows of blocks that were shared: a workgroup takes some heads of a token, DV / 4
// threads a row, and brings the parts' sums to the largest maximum.
template <typename T, int DV>
__global__ __launch_bounds__(THREADS) void latent_prefill_join_kernel(LatentPrefillArgs a, Parts split, int groups) {
  constexpr int WIDTH = DV / 4, HEADS = THREADS / WIDTH;
  const int t = blockIdx.x / groups, head = blockIdx.x % groups * HEADS + threadIdx.x / WIDTH;
  const int at = 4 * (threadIdx.x % WIDTH);
  const int n = a.cu ? find_last(a.n_seqs, [&](int i) { return seq_start(a.cu, i, a.q_total) <= t; }) : 0;
  const int q0 = a.cu ? seq_start(a.cu, n, a.q_total) : 0, q1 = a.cu ? seq_start(a.cu, n + 1, a.q_total) : a.q_total;
  if (t < q0 || t >= q1 || head >= a.n_heads) return;
  const int32_t* cu_k = a.cu_k ? a.cu_k : a.cu;
  const int k0 = cu_k ? seq_start(cu_k, n, a.k_total) : 0, k1 = cu_k ? seq_start(cu_k, n + 1, a.k_total) : a.k_total;
  const int past = max(k1 - k0, 0) - (q1 - q0);
  const int end = min((t - q0) / QB * QB + QB, q1 - q0) + past;
  const int all = end > 0 ? (end + KB - 1) / KB : 0, share = split.share(all);
  if (share >= all) return;
  const int parts = (all + share - 1) / share;
  const float c = a.scale * kLog2e;
  const int64_t place = (int64_t)t * a.n_heads + head, step = (int64_t)a.q_total * a.n_heads;
  float m = -__builtin_inff(), l = 0.f;
  f32x4 o = zero4();
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    const float2 st = split.stats[place + p * step];
    const f32x4 x = *reinterpret_cast<const f32x4*>(split.sums + (place + p * step) * DV + at);
    const float top = fmaxf(m, st.x), base = top == -__builtin_inff() ? 0.f : __fmul_rn(top, c);
    const float before = fast_exp2(__fmul_rn(m, c) - base), now = fast_exp2(__fmul_rn(st.x, c) - base);
    m = top;
    l = l * before + st.y * now;
    o = o * before + x * now;
  }
  const float inv = t - q0 + past >= 0 ? 1.f / l : 0.f;  // no key: O is 0
  typename Vec4<T>::type y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(o[e] * inv);
  *reinterpret_cast<typename Vec4<T>::type*>(static_cast<T*>(a.o) + (int64_t)t * a.o_stride + head * DV + at) = y;
}

template <typename T, int DN, int DR, int DV>
hipError_t run(const LatentPrefillArgs& a, const Parts& split, hipStream_t stream) {
  const int64_t blocks = latent_query_blocks(a.q_total, a.n_seqs);
  int classes = 1;  // of heads: the XCDs share them evenly
  while (classes < 8 && a.n_heads % (2 * classes) == 0) classes *= 2;
  const int64_t per = 8 / classes;
  const int64_t grid = 8 * ((blocks + per - 1) / per) * (a.n_heads / classes) * split.parts;
  const hipError_t e =
      enqueue(latent_prefill_kernel<T, DN, DR, DV>, (unsigned)grid, THREADS, stream, a, split, (int)blocks, classes);
  if (e != hipSuccess || split.parts == 1) return e;
  const int groups = (a.n_heads + THREADS / (DV / 4) - 1) / (THREADS / (DV / 4));
  return enqueue(latent_prefill_join_kernel<T, DV>, (unsigned)(a.q_total * groups), THREADS, stream, a, split, groups);
}

template <typename T, int DN, int DR>
hipError_t by_dv(const LatentPrefillArgs& a, const Parts& s, hipStream_t stream) {
  return a.dv == 128 ? run<T, DN, DR, 128>(a, s, stream) : run<T, DN, DR, 64>(a, s, stream);
}

template <typename T, int DN>
hipError_t by_dr(const LatentPrefillArgs& a, const Parts& s, hipStream_t stream) {
  return a.dr == 64 ? by_dv<T, DN, 64>(a, s, stream) : by_dv<T, DN, 32>(a, s, stream);
}

template <typename T>
hipError_t by_dn(const LatentPrefillArgs& a, const Parts& s, hipStream_t stream) {
  return a.dn == 128 ? by_dr<T, 128>(a, s, stream) : by_dr<T, 64>(a, s, stream);
}

int64_t sums_bytes(const LatentPrefillArgs& a, int parts) { return (int64_t)parts * a.q_total * a.n_heads * a.dv * 4; }

}  // namespace

size_t latent_prefill_workspace_bytes(const LatentPrefillArgs& a) {
  const int parts = a.q_total == 0 ? 1 : parts_of(a);
  return parts == 1 ? 0 : (size_t)(sums_bytes(a, parts) + (int64_t)parts * a.q_total * a.n_heads * 8);
}

hipError_t launch_latent_prefill(const LatentPrefillArgs& a, void* workspace, hipStream_t stream) {
  if (a.q_total == 0) return hipSuccess;
  Parts s = {parts_of(a), static_cast<float*>(workspace), nullptr};
  if (s.parts > 1) s.stats = reinterpret_cast<float2*>(static_cast<char*>(workspace) + sums_bytes(a, s.parts));
  return a.bf16 ? by_dn<bf16>(a, s, stream) : by_dn<float>(a, s, stream);
}

}  // namespace kda
