// kda_latent_attend.hip -- absorbed latent attention over a paged cache
// (kda_latent_attend): new tokens' queries of all heads against the cached rows
// [c | k_pe] themselves, o = sum_j p_j c_j.
//
// All heads share the rows, so a row of queries is a (token, head) pair and a
// workgroup takes 32 of a sequence's (a unit).  It walks the rows of the cache in
// tiles of 64 through LDS, where a tile is keys and values at once.  Four waves
// share a tile's work: for the scores S^T = C Q^T each takes 16 keys (and keeps all
// its queries' fragments in registers), for O^T += C^T P^T a quarter of the dc
// columns; the weights P and the maxima are exchanged through LDS.
//
// The tiles of all units together are cut into equal runs, one per workgroup, so
// that a long sequence is read by many.  A unit that is cut leaves its pieces
// (unnormalised sums, maximum, sum of weights, fp32) in the workspace and
// latent_join_kernel adds them up.
#include "kda_enqueue.h"
#include "kda_latent_launch.h"
#include "kda_latent_ops.h"

namespace kda {
namespace {

constexpr int KB = 64, THREADS = 256, ROWS = 32;
constexpr int RUNS = 256;      // workgroups: a tile of 64 x 576 in LDS leaves room for one per CU
constexpr int MIN_TILES = 2;   // of a run

// Units of a call at most, and the workspace: a head per unit, then pieces.  A run
// has at most two pieces of units that are cut: one that begins inside its unit
// (place 2 run) and one that begins with it (2 run + 1).
struct Plan {
  int64_t units;
  int runs;
  size_t heads_bytes, sums_bytes, bytes;
  Plan(int64_t t_total, int64_t n_seqs, bool one_each, int64_t n_heads, int dc, int64_t capacity) {
    units = one_each ? n_seqs * ((n_heads + ROWS - 1) / ROWS) : t_total * n_heads / ROWS + n_seqs;
    const int64_t tiles = units * ((capacity + KB - 1) / KB);
    runs = (int)(tiles < RUNS ? (tiles < 1 ? 1 : tiles) : RUNS);
    heads_bytes = ((size_t)units * sizeof(int2) + 255) / 256 * 256;
    sums_bytes = (size_t)runs * 2 * ROWS * dc * 4;
    bytes = heads_bytes + sums_bytes + (size_t)runs * 2 * ROWS * 8;
  }
  Plan(const LatentAttendArgs& a)
      : Plan(a.pages.t_total, a.pages.n_seqs, !a.pages.cu, a.n_heads, a.dc,
             (int64_t)a.pages.max_pages * a.pages.page_size) {}
};

struct Workspace {
  int2* heads;   // per unit: the run of its first piece, and how many more follow (0: not cut)
  float* sums;   // [2 runs][ROWS][dc]
  float2* stats; // [2 runs][ROWS]: maximum (of scores), sum of weights (-1: nothing seen)
};

// What a call's sequence holds.
struct Sequence {
  int start, tokens;        // first new token; new tokens
  int length, rows;         // seq_lens, and the rows of it that the table has places for
  int64_t units;
  int tiles;  // of each unit (one at least)
};
__device__ __forceinline__ Sequence sequence_of(const LatentPages& g, int n_heads, int n) {
  Sequence s;
  s.start = seq_start(g.cu, n, g.t_total);
  s.tokens = max((g.cu ? seq_start(g.cu, n + 1, g.t_total) : n + 1) - s.start, 0);
  s.length = max(g.lens[n], 0);
  s.rows = min(s.length, g.max_pages * g.page_size);
  s.units = ((int64_t)s.tokens * n_heads + ROWS - 1) / ROWS;
  s.tiles = max((s.rows + KB - 1) / KB, 1);
  return s;
}

// Inclusive sum over the workgroup's threads.
__device__ __forceinline__ int64_t scan(int64_t x, int64_t* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  for (int w = 0; w < wave; ++w) x += waves[w];
  return x;
}

template <typename T, int DC, int DR>
struct Shape {
  static constexpr int ES = sizeof(T), W = DC + DR;
  static constexpr int blocks = (W * ES + 127) / 128;   // column blocks of a row
  static constexpr int tile = blocks * KB * 128;
  static constexpr int p_row = KB * ES + 16;            // bytes of a row of weights
};

template <typename T, int DC, int DR>
__global__ __launch_bounds__(THREADS, 1) void latent_attend_kernel(LatentAttendArgs a, Workspace ws) {
  using S = Shape<T, DC, DR>;
  using F = typename Frag<T>::type;
  constexpr int ES = S::ES, W = S::W, KS = W / 32, NV = DC / 128, NT = ROWS / 16;
  __shared__ __attribute__((aligned(128))) char lds[S::tile];
  __shared__ __attribute__((aligned(16))) char weights[ROWS * S::p_row];
  __shared__ float tops[4][ROWS], sums[4][ROWS];
  __shared__ int seen_by[4][ROWS], odd_by[4];
  __shared__ int64_t waves[4], found[2];
  const LatentPages& g = a.pages;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int col = lane & 15, grp = lane >> 4;  // of a 16 x 16 tile

  // this workgroup's run of tiles, and the sequence it begins in
  const int run = blockIdx.x;
  int64_t total = 0, mine = 0;
  for (int base = 0; base < g.n_seqs; base += THREADS) {
    const int n = base + threadIdx.x;
    int64_t x = 0;
    if (n < g.n_seqs) {
      const Sequence s = sequence_of(g, a.n_heads, n);
      x = s.units * s.tiles;
    }
    mine = scan(x, waves);
    __syncthreads();
    if (threadIdx.x == THREADS - 1) found[0] = mine;
    __syncthreads();
    total += found[0];
  }
  const int runs = (int)min((int64_t)gridDim.x, max(total / MIN_TILES, (int64_t)1));
  const auto bound = [&](int64_t r) { return total * r / runs; };
  if (run >= runs) return;
  const int64_t lo = bound(run), hi = bound(run + 1);
  if (lo >= hi) return;
  int64_t before = 0;
  for (int base = 0;; base += THREADS) {
    const int n = base + threadIdx.x;
    int64_t x = 0;
    if (n < g.n_seqs) {
      const Sequence s = sequence_of(g, a.n_heads, n);
      x = s.units * s.tiles;
    }
    const int64_t upto = before + scan(x, waves);
    if (x > 0 && upto - x <= lo && lo < upto) {
      found[0] = n;
      found[1] = upto - x;
    }
    __syncthreads();
    if (threadIdx.x == THREADS - 1) waves[0] = upto;
    __syncthreads();
    before = waves[0];
    if (lo < before) break;
  }
  int n = (int)found[0];
  int64_t seq_at = found[1];  // the tile that the sequence's first unit begins with
  const float c = a.scale * kLog2e;

  for (int64_t pos = lo; pos < hi;) {
    const Sequence s = sequence_of(g, a.n_heads, n);
    const int64_t in_seq = pos - seq_at;
    const int unit = (int)(in_seq / s.tiles), tile0 = (int)(in_seq - (int64_t)unit * s.tiles);
    const int tile1 = (int)min((int64_t)s.tiles, tile0 + (hi - pos));
    const int64_t unit_at = pos - tile0;
    pos += tile1 - tile0;
    const int n_now = n;
    if (pos - seq_at == s.units * s.tiles) {
      seq_at = pos;
      ++n;
      while (pos < hi && n + 1 < g.n_seqs && sequence_of(g, a.n_heads, n).units == 0) ++n;
    }

    // the unit's queries: row r is head (r % H) of new token r / H; it sees positions
    // below limit(r)
    const int row0 = unit * ROWS, n_rows = s.tokens * a.n_heads;
    const auto limit_of = [&](int r) {
      const int tok = min(row0 + r, n_rows - 1) / a.n_heads;
      return min(max(s.length + (tok + 1 - s.tokens), 0), s.rows);
    };
    const int most = limit_of(ROWS - 1), least = limit_of(0);
    F q[NT][KS];
    int limit[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = min(row0 + 16 * t + col, n_rows - 1), tok = r / a.n_heads;
      const T* qr = static_cast<const T*>(a.q) + (s.start + tok) * a.q_stride + (int64_t)(r - tok * a.n_heads) * W;
      limit[t] = limit_of(16 * t + col);
#pragma unroll
      for (int k = 0; k < KS; ++k) q[t][k] = load_frag8<T>(qr + 32 * k + 8 * grp);
    }
    const int my_limit = limit_of(lane & 31);  // of the query whose output this lane holds
    f32x16 o[NV];
#pragma unroll
    for (int d = 0; d < NV; ++d) o[d] = zero16();
    float top[NT], sum[NT], top_o = -__builtin_inff();
    bool seen[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) top[t] = -__builtin_inff(), sum[t] = 0.f, seen[t] = false;

    const int tiles_end = min(tile1, (most + KB - 1) / KB);
    for (int tile = tile0; tile < tiles_end; ++tile) {
      // rows 16 wave .. 16 wave + 15 of the tile: eight lanes to a row's 128 bytes.  A
      // position without a row is 0 and not seen.
      const int j0 = tile * KB;
      uint64_t have[2];
      __syncthreads();
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * wave + 8 * r + (lane >> 3), j = j0 + row, chunk = lane & 7;
        int page = -1;
        if (j < s.rows) page = g.table[(int64_t)n_now * g.max_pages + j / g.page_size];
        const bool in = page >= 0 && page < g.n_pages;
        have[r] = __ballot(in);
        const char* src = static_cast<const char*>(a.cache) +
                          ((int64_t)(in ? page : 0) * g.page_stride + (j % g.page_size) * g.row_stride) * ES + chunk * 16;
#pragma unroll
        for (int b = 0; b < S::blocks; ++b) {
          uint4 x = {0, 0, 0, 0};
          if (in && b * 128 + chunk * 16 < W * ES) x = *reinterpret_cast<const uint4*>(src + b * 128);
          *reinterpret_cast<uint4*>(lds + b * KB * 128 + tile_at<KB>(row, chunk * 16)) = x;
        }
      }
      __syncthreads();

      // scores of this wave's keys: element i of a lane is key 4 grp + i
      f32x4 x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t] = zero4();
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const F key = tile_row8<KB>(lds, 16 * wave + col, 32 * k + 8 * grp, T());
#pragma unroll
        for (int t = 0; t < NT; ++t) x[t] = mma32(key, q[t][k], x[t]);
      }
      bool odd = false;  // a score that is not finite of a key that some query does not see
      const uint64_t have_mine = grp < 2 ? have[0] : have[1];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        float mx = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool sees = j0 + 16 * wave + 4 * grp + i < limit[t] && (have_mine >> (8 * (4 * (grp & 1) + i)) & 1);
          odd |= !sees && !__builtin_isfinite(x[t][i]);
          seen[t] |= sees;
          if (!sees) x[t][i] = -__builtin_inff();
          mx = fmaxf(mx, x[t][i]);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (grp == 0) tops[wave][16 * t + col] = mx;
      }
      odd = __any(odd);
      if (lane == 0) odd_by[wave] = odd;
      __syncthreads();
      const auto tops_of = [&](int r, float m) {
        return fmaxf(m, fmaxf(fmaxf(tops[0][r], tops[1][r]), fmaxf(tops[2][r], tops[3][r])));
      };
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float m = tops_of(16 * t + col, top[t]);
        const float base = m == -__builtin_inff() ? 0.f : __fmul_rn(m, c);
        sum[t] *= fast_exp2(__fmul_rn(top[t], c) - base);
        top[t] = m;
        typename Vec4<T>::type p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = fast_exp2(x[t][i] * c - base);
          sum[t] += e;
          p[i] = from_f32<T>(e);  // bf16: one rounding, 2^-8
        }
        *reinterpret_cast<typename Vec4<T>::type*>(weights + (16 * t + col) * S::p_row + (16 * wave + 4 * grp) * ES) = p;
      }
      const float m = tops_of(lane & 31, top_o);
      const float alpha = fast_exp2(__fmul_rn(top_o, c) - (m == -__builtin_inff() ? 0.f : __fmul_rn(m, c)));
      top_o = m;
      if (__any(alpha != 1.f)) {
#pragma unroll
        for (int d = 0; d < NV; ++d) o[d] *= alpha;
      }
      const bool special = j0 + KB > least && (odd_by[0] | odd_by[1] | odd_by[2] | odd_by[3]);
      __syncthreads();

      // O^T of this wave's columns
      F p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const char* row = weights + (lane & 31) * S::p_row + (16 * k + 4 * h) * ES;
        const auto lo4 = *reinterpret_cast<const typename Vec4<T>::type*>(row);
        const auto hi4 = *reinterpret_cast<const typename Vec4<T>::type*>(row + 8 * ES);
#pragma unroll
        for (int e = 0; e < 4; ++e) p[k][e] = lo4[e], p[k][4 + e] = hi4[e];
      }
      if (!special) {
#pragma unroll
        for (int d = 0; d < NV; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            o[d] = mma16(tile_col8<KB>(lds, 16 * k, (DC / 4) * wave + 32 * d, lane, T()), p[k], o[d]);
      } else {
#pragma unroll
        for (int d = 0; d < NV; ++d) {
          f32x16 kinds = zero16();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            F v = tile_col8<KB>(lds, 16 * k, (DC / 4) * wave + 32 * d, lane, T()), kind, sees;
            split_special(v, kind);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              sees[e] = from_f32<T>(j0 + 16 * k + 8 * (e >> 2) + 4 * h + (e & 3) < my_limit ? 1.f : 0.f);
            o[d] = mma16(v, p[k], o[d]);
            kinds = mma16(kind, sees, kinds);
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] = add_special(o[d][i], kinds[i]);
        }
      }
    }

    // the sum of weights of each row, over lanes and waves
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x = sum[t];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      int any = seen[t];
      any |= __shfl_xor(any, 16);
      any |= __shfl_xor(any, 32);
      if (grp == 0) sums[wave][16 * t + col] = x, seen_by[wave][16 * t + col] = any;
    }
    __syncthreads();
    const int r = lane & 31;
    const float all = (sums[0][r] + sums[1][r]) + (sums[2][r] + sums[3][r]);
    const bool some = seen_by[0][r] | seen_by[1][r] | seen_by[2][r] | seen_by[3][r];
    if (tile0 == 0) {
      // the unit's last piece is in the last run that begins before the unit ends
      const int more = (int)(((unit_at + s.tiles) * runs + total - 1) / total) - 1 - run;
      if (threadIdx.x == 0) {
        const int64_t id = g.cu ? first_block<ROWS>(s.start, a.n_heads, n_now) : (int64_t)n_now * s.units;
        ws.heads[id + unit] = int2{run, more};
      }
    }
    if (tile0 == 0 && tile1 == s.tiles) {
      if (row0 + r < n_rows) {
        const int tok = (row0 + r) / a.n_heads;
        const float inv = some ? 1.f / all : 0.f;  // no key: O is 0
        T* out = static_cast<T*>(a.o) + (s.start + tok) * a.o_stride + (int64_t)(row0 + r - tok * a.n_heads) * DC +
                 (DC / 4) * wave;
#pragma unroll
        for (int d = 0; d < NV; ++d)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            typename Vec4<T>::type y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(o[d][4 * b + e] * inv);
            *reinterpret_cast<typename Vec4<T>::type*>(out + 32 * d + 8 * b + 4 * h) = y;
          }
      }
    } else {
      const int64_t place = 2 * (int64_t)run + (tile0 == 0 ? 1 : 0);
      float* out = ws.sums + (place * ROWS + r) * DC + (DC / 4) * wave;
#pragma unroll
      for (int d = 0; d < NV; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<f32x4*>(out + 32 * d + 8 * b + 4 * h) =
              f32x4{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
      if (wave == 0 && lane < 32) ws.stats[place * ROWS + r] = float2{top_o, some ? all : -1.f};
    }
  }
}

// A row of a unit that was cut: the pieces' sums, each at its own maximum, brought to
// the largest.  A thread takes four columns.
template <typename T, int DC>
__global__ __launch_bounds__(DC / 4) void latent_join_kernel(LatentAttendArgs a, Workspace ws) {
  const LatentPages& g = a.pages;
  const int64_t id = blockIdx.x / ROWS;
  const int r = blockIdx.x % ROWS;
  int n;
  int64_t unit;
  if (g.cu) {
    n = find_sequence<ROWS>(g.cu, g.n_seqs, g.t_total, a.n_heads, id);
    unit = id - first_block<ROWS>(seq_start(g.cu, n, g.t_total), a.n_heads, n);
  } else {
    const int64_t per = (a.n_heads + ROWS - 1) / ROWS;
    n = (int)(id / per);
    unit = id - n * per;
  }
  const Sequence s = sequence_of(g, a.n_heads, n);
  if (unit < 0 || unit >= s.units) return;
  const int64_t row = unit * ROWS + r;
  if (row >= (int64_t)s.tokens * a.n_heads) return;
  const int2 head = ws.heads[id];
  if (head.y == 0) return;
  const float c = a.scale * kLog2e;
  const auto place = [&](int i) { return ((int64_t)(i == 0 ? 2 * head.x + 1 : 2 * (head.x + i)) * ROWS + r); };
  float top = -__builtin_inff();
  for (int i = 0; i <= head.y; ++i) {
    const float2 st = ws.stats[place(i)];
    if (!(st.y == -1.f)) top = fmaxf(top, st.x);
  }
  const float base = top == -__builtin_inff() ? 0.f : __fmul_rn(top, c);
  f32x4 o = zero4();
  float sum = 0.f;
  bool some = false;
  for (int i = 0; i <= head.y; ++i) {
    const float2 st = ws.stats[place(i)];
    if (st.y == -1.f) continue;
    some = true;
    const float f = fast_exp2(__fmul_rn(st.x, c) - base);
    sum += f * st.y;
    o += f * *reinterpret_cast<const f32x4*>(ws.sums + place(i) * DC + 4 * threadIdx.x);
  }
  const float inv = some ? 1.f / sum : 0.f;
  const int tok = (int)(row / a.n_heads);
  T* out = static_cast<T*>(a.o) + (s.start + tok) * a.o_stride + (row - (int64_t)tok * a.n_heads) * DC + 4 * threadIdx.x;
  typename Vec4<T>::type y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(o[e] * inv);
  *reinterpret_cast<typename Vec4<T>::type*>(out) = y;
}

template <typename T, int DC, int DR>
hipError_t run(const LatentAttendArgs& a, const Plan& plan, const Workspace& ws, hipStream_t stream) {
  hipError_t e = enqueue(latent_attend_kernel<T, DC, DR>, (unsigned)plan.runs, THREADS, stream, a, ws);
  if (e != hipSuccess) return e;
  return enqueue(latent_join_kernel<T, DC>, (unsigned)(plan.units * ROWS), DC / 4, stream, a, ws);
}

template <typename T>
hipError_t by_shape(const LatentAttendArgs& a, const Plan& plan, const Workspace& ws, hipStream_t stream) {
  if (a.dc == 512) return a.dr == 64 ? run<T, 512, 64>(a, plan, ws, stream) : run<T, 512, 32>(a, plan, ws, stream);
  return a.dr == 64 ? run<T, 256, 64>(a, plan, ws, stream) : run<T, 256, 32>(a, plan, ws, stream);
}

}  // namespace

size_t latent_workspace_bytes(const LatentAttendArgs& a) {
  return a.pages.t_total == 0 || a.pages.n_seqs == 0 ? 0 : Plan(a).bytes;
}

hipError_t launch_latent_attend(const LatentAttendArgs& a, void* workspace, hipStream_t stream) {
  if (a.pages.t_total == 0 || a.pages.n_seqs == 0) return hipSuccess;
  const Plan plan(a);
  char* w = static_cast<char*>(workspace);
  const Workspace ws = {reinterpret_cast<int2*>(w), reinterpret_cast<float*>(w + plan.heads_bytes),
                        reinterpret_cast<float2*>(w + plan.heads_bytes + plan.sums_bytes)};
  return a.bf16 ? by_shape<bf16>(a, plan, ws, stream) : by_shape<float>(a, plan, ws, stream);
}

}  // namespace kda
