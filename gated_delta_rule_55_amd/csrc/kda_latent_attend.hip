// kda_latent_attend.hip -- absorbed latent attention over a paged cache
// (kda_latent_attend): new tokens' queries of all heads against the cached rows
// [c | k_pe] themselves, o = sum_j p_j c_j, p the softmax of scale q . row_j.
//
// All heads share the rows, so a row of queries is a (token, head) pair and a
// workgroup takes R = 32 or 64 of a sequence's (a unit).  It walks the rows of the
// cache in tiles (bf16 64 rows, fp32 32) through LDS, where a tile is keys and values
// at once; two tiles, one worked on while the other is fetched straight into LDS, fill
// it, so a CU has one workgroup (bf16 eight waves, fp32 four).  Waves share a tile's
// work: for the scores S^T = C Q^T they are R / 16 groups of queries, whose
// fragments they keep in registers, times groups of keys; for O^T += C^T P^T each
// has its share of the dc columns, in registers from the first tile to the last.  The
// maxima and the weights P are exchanged through LDS; running maxima and sums are
// fp32, and O is scaled only by tiles that raise a maximum.
//
// The tiles of all units together are cut into equal runs, one per workgroup, so
// that a long sequence is read by many.  A unit that is cut leaves its pieces
// (unnormalised sums, maximum, sum of weights, fp32) in the workspace and
// latent_join_kernel adds them up.
//
// What bounds it (512 + 64, bf16).  One token a sequence: the rows' bytes; 64 sequences of
// 8,192 rows on average, 32 heads, 137 us, 4.4 TB/s of the 5.0 that a copy reaches.  Many queries a row:
// a tile's turn takes 2.8 us at R = 64, of which the matrix instructions are 0.9, the
// reads of LDS (each key by four waves) 1.4, and three barriers keep the two from
// overlapping fully: 2,048 new tokens of 32 heads on 18,432 rows 3.1 ms, 0.81 PFLOP/s.  A few
// tokens a sequence: the rows' bytes again, but a sequence's two or three units take its rows at
// different times on different XCDs, so that 24 sequences of 113 MB read 343 and write 60 of
// pieces, at 4.7 TB/s.  One sequence of 32,768 rows, 28 us: a piece's start (tables, pages and
// first rows one after the other) and end 11, four tiles of 1.9, the join and its launch 6, and 4
// for what 128 workgroups at once have to wait for the memory.
//
// In bf16 the weights P are rounded before they meet the values (2^-8 of a weight at most), since
// the matrix cores take operands of one type and fp32's run at an eighth of the rate; a second
// product for the rest of each weight would double the work of O.  Their sum is taken before
// that.  Against float64 the outputs' error grows from that of their own rounding, 1.7e-3 of
// their norm, to 1.8e-3.
//
// Every unit counts as all of its sequence's rows where the tiles are shared out, though its
// queries may see fewer: where the new tokens are most of the sequence, the runs of its first
// units are done early (2,048 new tokens of 2,048 rows: the longest walks 128 tiles, the mean 66).
#include "kda_enqueue.h"
#include "kda_latent_launch.h"
#include "kda_latent_ops.h"

namespace kda {
namespace {

constexpr int JOIN_THREADS = 256;
constexpr int RUNS = 256;     // workgroups: their tiles in LDS leave room for one per CU
// What it costs to begin a unit's piece (its queries, the first rows' latency) and to end
// it, in tiles of KB rows (64: bf16; fp32's 32 rows take longer, 5 us: three sequences of 200
// rows 26 us with 1, 30 with 2, 41 with 3): each unit counts as that many more, in front, so
// that a run that crosses from one into another has fewer tiles for it.
constexpr int setup_of(int KB) { return KB == 64 ? 3 : 1; }
// Tiles of a run at least, a unit's setup among them where the run begins one; a run inside a unit
// has this many of the unit's.  Half of these would give a short sequence more workgroups and a
// long one more pieces to join.  bf16, 32 heads, one sequence, us for 4 / 2 / 1: 1,000 rows 24.0 /
// 18.7 / 17.2, 8,192 rows 24.5 / 20.9 / 21.9, 32,768 rows 28.6 / 30.9 / 30.9, 131,072 rows and
// batches of 8 and more sequences the same; 5: 1,000 rows 27 for 25, 32,768 rows 30 both ways.
// fp32: three sequences of 200 rows 25.0 us, with 1 19.6.
constexpr int min_tiles(int KB) { return setup_of(KB) + 1; }

// The workspace.  A run has at most two pieces of units that are cut: one that begins
// inside its unit (place 2 run) and one that begins with it (place 2 run + 1).  The
// latter's head says where the unit's other pieces are.  Heads are numbered by unit
// where a call has few of them, so that the join has a workgroup for each row of these and
// no idle ones (one sequence of 32,768 rows, 128 heads: 46 us, by run 69), else by run,
// with 16 workgroups each, which idle where a run begins no unit that is cut (by unit and by
// run, us: 16 units 33.9 and 35.8, 64 sequences of 4,000 rows 75.3 and 77.0, of 300 rows 26.9 and
// 29.2; 128 of 2,000 rows 82.3 and 84.2, 256 of 1,000 rows 68.8 and 67.8).  Where even the
// rows would not fill the GPU a workgroup takes 128 columns of one (columns by 128 and whole rows,
// us: 1 unit 28.6 and 33.2, 8 units 32.4 and 33.5, 16 units 33.9 both ways, 32 units 45.7 and 43.9,
// 64 units 80.9 and 75.0).
constexpr int FEW_UNITS = 64, JOIN_SHARES = 16;
// Units are of 64 rows where that leaves a run this many tiles, as far as the host can tell: lengths
// are on the device, and each sequence counts as long as the table has places.  Each is read from LDS
// and from memory half as often (2,048 new tokens 3.0 ms for 4.6, 24 sequences of some 4
// tokens 93 us for 108, 256
// sequences of 1,000 rows and 128 heads 166 for 225).  With fewer tiles the shorter turns of
// 32 rows, in more runs, win (four sequences of 8,000 rows, 128 heads: 40 us for 50).
constexpr int LONG_RUN = 6;
struct Plan {
  int rows;  // of a unit
  bool by_unit;
  int64_t units;  // at most
  int runs, heads;
  size_t heads_bytes, sums_bytes, bytes;
  explicit Plan(const LatentAttendArgs& a) {
    const int64_t T = a.pages.t_total, N = a.pages.n_seqs, H = a.n_heads;
    const int tile = a.bf16 ? 64 : 32;
    const int64_t most = ((int64_t)a.pages.max_pages * a.pages.page_size + tile - 1) / tile;  // of a sequence
    rows = a.bf16 && T * H >= 64 * N && T * H / 64 * most >= LONG_RUN * RUNS ? 64 : 32;
    units = a.pages.cu ? T * H / rows + N : N * ((H + rows - 1) / rows);
    const int64_t tiles = units * (setup_of(tile) + most) / min_tiles(tile);
    runs = (int)(tiles < RUNS ? (tiles < 1 ? 1 : tiles) : RUNS);
    by_unit = units <= FEW_UNITS;
    heads = by_unit ? (int)units : runs;
    heads_bytes = ((size_t)heads * sizeof(int4) + 255) / 256 * 256;
    sums_bytes = (size_t)runs * 2 * rows * a.dc * 4;
    bytes = heads_bytes + sums_bytes + (size_t)runs * 2 * rows * 8;
  }
};

struct Workspace {
  int4* heads;    // run of the unit's first piece, how many more follow (0: not cut), first row, rows
  float* sums;    // [2 runs][R][dc]
  float2* stats;  // [2 runs][R]: maximum (of scores), sum of weights (-1: nothing seen)
  int by_unit;
};

// What a call's sequence holds.
struct Sequence {
  int start, tokens;        // first new token; new tokens
  int length, rows;         // seq_lens, and the rows of it that the table has places for
  int64_t units;            // of R queries
  int tiles;                // of KB rows, of each unit, and its setup
  __device__ __forceinline__ int64_t all() const { return units * tiles; }
};
template <int R, int KB>
__device__ __forceinline__ Sequence sequence_of(const LatentPages& g, int n_heads, int n) {
  Sequence s;
  s.start = seq_start(g.cu, n, g.t_total);
  s.tokens = max((g.cu ? seq_start(g.cu, n + 1, g.t_total) : n + 1) - s.start, 0);
  s.length = max(g.lens[n], 0);
  s.rows = min(s.length, g.max_pages * g.page_size);
  s.units = ((int64_t)s.tokens * n_heads + R - 1) / R;
  s.tiles = setup_of(KB) + max((s.rows + KB - 1) / KB, 1);
  return s;
}

// Inclusive sum over the workgroup's threads, and the sum of all.
template <int WAVES>
__device__ __forceinline__ int64_t scan(int64_t x, int64_t* waves, int64_t* all) {
  const int lane = threadIdx.x & 63, wave = wave_index();
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) waves[wave] = x;
  __syncthreads();
  *all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    if (w < wave) x += waves[w];
    *all += waves[w];
  }
  return x;
}

// a / b, in 32 bits where they do.
__device__ __forceinline__ int64_t divide(int64_t a, int b) {
  return a >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The tiles of all units (and their setups), total, in `runs` equal runs: the first `longer` of them have
// one more than the others' `share`.
template <int KB>
struct Runs {
  int64_t total, share;
  int runs, longer;
  __device__ __forceinline__ Runs(int64_t all, int most) : total(all) {
    runs = (int)min((int64_t)most, max(all / min_tiles(KB), (int64_t)1));
    share = divide(all, runs);
    longer = (int)(all - share * runs);
  }
  __device__ __forceinline__ int64_t begin(int run) const { return share * run + min(run, longer); }
  // runs behind `run` that the next `rest` tiles reach into
  __device__ __forceinline__ int reached(int run, int rest) const {
    if (rest == 0) return 0;
    if (share >= rest) return 1;
    const int same = max(longer - (run + 1), 0), each = (int)share;
    if (rest <= (int64_t)same * (each + 1)) return (rest + each) / (each + 1);
    return same + (rest - same * (each + 1) + each - 1) / each;
  }
};

// How NW waves share a tile of KB cached rows and a unit of R queries.  Scores: KG
// groups of keys times RG groups of queries, a wave KT tiles of 16 x 16.
// Outputs: a wave COLS of the columns, NV x RV tiles of 32 x 32.
template <typename T, int DC, int DR, int R>
struct Shape {
  static constexpr int ES = sizeof(T), W = DC + DR;
  static constexpr int KB = sizeof(T) == 2 ? 64 : 32;   // two tiles fill LDS
  static constexpr int NW = sizeof(T) == 2 ? 8 : 4, THREADS = 64 * NW;
  static constexpr int RG = R / 16, KG = NW / RG, KT = KB / (16 * KG);
  static constexpr int COLS = DC / NW, NV = COLS / 32, RV = R / 32;
  static constexpr int KS = W / 32;                     // slices of a score's sum
  static constexpr int blocks = (W * ES + 127) / 128;   // column blocks of a row
  static constexpr int tile = blocks * KB * 128;
  static constexpr int p_row = KB * ES + 16;            // bytes of a row of weights
};

// Source of the rows that do not exist: as long as the longest row.
__device__ const uint4 kNoRow[(512 + 64) * 4 / 16] = {};

template <typename T, int DC, int DR, int R>
struct Attend {
  using S = Shape<T, DC, DR, R>;
  using F = typename Frag<T>::type;
  using V4 = typename Vec4<T>::type;
  static constexpr int ES = S::ES, KB = S::KB;

  // LDS that the waves exchange through
  struct Exchange {
    float tops[S::KG][R], sums[S::KG][R];
    int seen[S::KG][R], odd[S::NW];
    uint64_t have[2][KB / 8];  // per tile in LDS: which of its rows exist, 8 bits to a row
  };

  F q[S::KS];
  f32x16 o[S::NV][S::RV];
  int limit, my_limit[S::RV];  // of the queries whose scores and outputs this lane holds
  float top, sum, top_o[S::RV];
  bool seen;
  RowFrags<T, KB, 32> key_frags;
  ColFrags<T, KB> value_frags;

  __device__ __forceinline__ Attend(int lane, int wave)
      : top(-__builtin_inff()), sum(0.f), seen(false), key_frags(wave % S::KG * S::KT * 16 + (lane & 15), lane >> 4),
        value_frags(S::COLS * wave, lane) {
#pragma unroll
    for (int v = 0; v < S::RV; ++v) {
      top_o[v] = -__builtin_inff();
#pragma unroll
      for (int d = 0; d < S::NV; ++d) o[d][v] = zero16();
    }
  }

  // Whether every query of the unit sees all of the tile at j0.
  static __device__ __forceinline__ bool whole(const uint64_t* have, int j0, int least, int lane) {
    const bool all = __ballot(have[lane % (KB / 8)] == ~(uint64_t)0) == ~(uint64_t)0;
    return j0 + KB <= least && all;
  }

  // One tile: positions j0 .. j0 + KB - 1, its rows in `tile`.  Where not all of it is seen
  // each (key, query) is looked at, and false is returned if a key that is not seen holds
  // a value that is not finite (its score is not): SAFE then does the whole unit again.
  // fetch(b) fetches column block b of the next tile, between the score's steps (all at once
  // they would hold the waves up).
  template <bool SAFE, typename Fetch>
  __device__ __forceinline__ bool step(const char* tile, const uint64_t* have, char* weights, Exchange& x, int j0,
                                       int least, float c, int lane, int wave, Fetch fetch) {
    const bool not_whole = !whole(have, j0, least, lane);
    const int h = lane >> 5, col = lane & 15, grp = lane >> 4;
    const int kg = wave % S::KG, rg = wave / S::KG;
    const int key0 = kg * S::KT * 16, row = rg * 16 + col;
    f32x4 sc[S::KT], sd[S::KT];  // two sums each, so that products need not wait for one another
#pragma unroll
    for (int k = 0; k < S::KT; ++k) sc[k] = sd[k] = zero4();
    pipelined<F, S::KS * S::KT, 4>([&](int i) { return key_frags.load(tile, i / S::KT, 16 * (i % S::KT)); },
                                   [&](int i, F key) {
                                     f32x4& acc = i / S::KT % 2 ? sd[i % S::KT] : sc[i % S::KT];
                                     acc = mma32(key, q[i / S::KT], acc);
                                   },
                                   [&](int g) {
                                     constexpr int groups = (S::KS * S::KT + 3) / 4, each = (S::blocks + groups - 1) / groups;
#pragma unroll
                                     for (int b = g * each; b < (g + 1) * each && b < S::blocks; ++b) fetch(b);
                                   });
#pragma unroll
    for (int k = 0; k < S::KT; ++k) sc[k] += sd[k];
    // element i of a lane: key key0 + 16 k + 4 grp + i
    bool odd = false;  // a score that is not finite of a key that its query does not see
    if (__builtin_expect(not_whole, 0)) {
#pragma unroll
      for (int k = 0; k < S::KT; ++k) {
        const int key = key0 + 16 * k + 4 * grp;
        const uint32_t there = (uint32_t)(have[key >> 3] >> (8 * (key & 4)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool sees = j0 + key + i < limit && (there >> (8 * i) & 1);
          odd |= !sees && !__builtin_isfinite(sc[k][i]);
          seen |= sees;
          sc[k][i] = sees ? sc[k][i] : -__builtin_inff();
        }
      }
      odd = __any(odd);
    } else {
      seen = true;
    }
    float mx = -__builtin_inff();
#pragma unroll
    for (int k = 0; k < S::KT; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = fmaxf(mx, sc[k][i]);
    mx = max_halves(max_sixteens(mx));
    x.tops[kg][row] = mx;  // (four lanes the same)
    if (!SAFE) x.odd[wave] = odd;
    exchanged();
    const auto tops_of = [&](int r, float m) {
#pragma unroll
      for (int k = 0; k < S::KG; ++k) m = fmaxf(m, x.tops[k][r]);
      return m;
    };
    {
      const float m = tops_of(row, top);
      // (a maximum's product with c is rounded the same way each time it is formed)
      const float base = m == -__builtin_inff() ? 0.f : __fmul_rn(m, c);
      sum *= fast_exp2(__fmul_rn(top, c) - base);
      top = m;
#pragma unroll
      for (int k = 0; k < S::KT; ++k) {
        V4 p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = fast_exp2(sc[k][i] * c - base);
          sum += e;
          p[i] = from_f32<T>(e);  // bf16: one rounding, 2^-8 (see the top)
        }
        *reinterpret_cast<V4*>(weights + row * S::p_row + (key0 + 16 * k + 4 * grp) * ES) = p;
      }
    }
#pragma unroll
    for (int v = 0; v < S::RV; ++v) {
      const float m = tops_of(32 * v + (lane & 31), top_o[v]);
      const float alpha = fast_exp2(__fmul_rn(top_o[v], c) - (m == -__builtin_inff() ? 0.f : __fmul_rn(m, c)));
      top_o[v] = m;
      if (__builtin_expect(__any(alpha != 1.f), 0)) {
#pragma unroll
        for (int d = 0; d < S::NV; ++d) o[d][v] *= alpha;
      }
    }
    if (!SAFE && __builtin_expect(not_whole, 0)) {
      if (__any(x.odd[lane % S::NW])) return false;
    }
    const auto value = [&](int i) { return value_frags.load(tile, 16 * (i / S::NV), i % S::NV); };
    F first[2];  // (read while the others come: 3.05 -> 3.01 ms)
#pragma unroll
    for (int i = 0; i < 2; ++i) first[i] = value(i);
    exchanged();

    const auto weight = [&](int v, int k) {
      const char* from = weights + (32 * v + (lane & 31)) * S::p_row + (16 * k + 4 * h) * ES;
      const V4 lo = *reinterpret_cast<const V4*>(from), hi = *reinterpret_cast<const V4*>(from + 8 * ES);
      F p;
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = lo[e], p[4 + e] = hi[e];
      return p;
    };
    if (SAFE && not_whole) {
      values_special(tile, weight, j0, lane);
      return true;
    }
    // step k NV + d: columns 32 d, rows 16 k of the tile, and their weights with d = 0
    F p[2][S::RV];
#pragma unroll
    for (int v = 0; v < S::RV; ++v) p[0][v] = weight(v, 0);
    pipelined_from<F, KB / 16 * S::NV, 2>(
        first, value,
        [&](int i, F val) {
          const int k = i / S::NV, d = i % S::NV;
          if (d == 0 && k + 1 < KB / 16) {
#pragma unroll
            for (int v = 0; v < S::RV; ++v) p[(k + 1) % 2][v] = weight(v, k + 1);
          }
#pragma unroll
          for (int v = 0; v < S::RV; ++v) o[d][v] = mma16(val, p[k % 2][v], o[d][v]);
        },
        [](int) {});
    return true;
  }

  template <typename Weight>
  __device__ __forceinline__ void values_special(const char* tile, Weight weight, int j0, int lane) {
    const int h = lane >> 5;
#pragma unroll
    for (int d = 0; d < S::NV; ++d)
#pragma unroll
      for (int v = 0; v < S::RV; ++v) {
        f32x16 kinds = zero16();
#pragma unroll
        for (int k = 0; k < KB / 16; ++k) {
          F val = value_frags.load(tile, 16 * k, d), kind, sees;
          split_special(val, kind);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sees[e] = from_f32<T>(j0 + 16 * k + 8 * (e >> 2) + 4 * h + (e & 3) < my_limit[v] ? 1.f : 0.f);
          o[d][v] = mma16(val, weight(v, k), o[d][v]);
          kinds = mma16(kind, sees, kinds);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][v][i] = add_special(o[d][v][i], kinds[i]);
      }
  }
};

// What a workgroup does of a unit: tiles tile0 .. tile1 - 1 of it.
struct Piece {
  int n, unit, tile0, tile1;
  int run, more;  // the run this is of, and how many behind it have the unit's rest
};

template <typename T, int DC, int DR, int R, bool SAFE>
__device__ __forceinline__ bool attend_piece(const LatentAttendArgs& a, const Workspace& ws, const Sequence& s,
                                             const Piece& pc, char* even, char* odd, char* weights,
                                             typename Attend<T, DC, DR, R>::Exchange& x) {
  using S = Shape<T, DC, DR, R>;
  using A = Attend<T, DC, DR, R>;
  constexpr int ES = S::ES, W = S::W, KB = S::KB;
  const LatentPages& g = a.pages;
  const int lane = threadIdx.x & 63, wave = wave_index(), h = lane >> 5;
  const int col = lane & 15, grp = lane >> 4;  // of a 16 x 16 tile
  const float c = a.scale * kLog2e;
  const int unit = pc.unit, tile0 = pc.tile0, tile1 = pc.tile1, n_now = pc.n, run = pc.run;
  // the unit's queries: row r is head (r % H) of new token r / H; it sees positions
  // below limit(r)
  const int row0 = unit * R, n_rows = s.tokens * a.n_heads;
  const auto limit_of = [&](int r) {
    const int tok = min(row0 + r, n_rows - 1) / a.n_heads;
    return min(max(s.length + (tok + 1 - s.tokens), 0), s.rows);
  };
  const int most = limit_of(R - 1), least = limit_of(0);
  const int tiles_end = min(tile1, (most + KB - 1) / KB);

  // The next tile is fetched while one is worked on, and the pages of the one after
  // that looked up.  A wave fetches eight rows, eight lanes to 128 bytes of a row, the
  // chunks exchanged as tile_at has them; a position without a row is 0 and not seen.
  static_assert(KB == 8 * S::NW, "a wave fetches eight rows of a tile");
  const int fetch_row = 8 * wave + (lane >> 3), chunk = ((lane & 7) ^ row_swap(lane >> 3)) * 16;
  int page = -1;
  const char* from;
  const int32_t* const pages = g.table + (int64_t)n_now * g.max_pages;
  const auto look_up = [&](int tile) {
    const int j = tile * KB + fetch_row;
    const int p = pages[min(page_of(g, j), g.max_pages - 1)];
    page = tile < tiles_end && j < s.rows ? p : -1;
  };
  // the rows of `tile`, whose pages have been looked up; those of the tile behind it
  const auto aim = [&](int tile, uint64_t* have) {
    const int j = tile * KB + fetch_row;
    const bool in = page >= 0 && page < g.n_pages;
    have[wave] = __ballot(in);
    const int64_t at = (int64_t)page * g.page_stride + row_in_page(g, j, page_of(g, j)) * g.row_stride;
    const char* const row = static_cast<const char*>(a.cache) + at * ES;
    from = (in ? row : reinterpret_cast<const char*>(kNoRow)) + chunk;
    look_up(tile + 1);
  };
  // column block b of them, one after the other
  const auto fetch = [&](int b, char* to) {
    const char* p = from;
    if (128 * (b + 1) > W * ES && 128 * b + chunk >= W * ES) p = reinterpret_cast<const char*>(kNoRow);
    fetch16(p, to + (b * KB + 8 * wave) * 128);
    if (b + 1 < S::blocks) from = next_line(from);
  };

  A s_(lane, wave);
  look_up(tile0);
  // LDS of the piece before is done with (where that stopped, a tile's fetches too)
  if (SAFE)
    fetched();
  else
    exchanged();
  aim(tile0, x.have[0]);
#pragma unroll
  for (int b = 0; b < S::blocks; ++b) fetch(b, even);
  // (the queries come while the rows do)
  const int kg = wave % S::KG, rg = wave / S::KG;
  {
    const int r = min(row0 + rg * 16 + col, n_rows - 1), tok = r / a.n_heads;
    const T* qr = static_cast<const T*>(a.q) + (s.start + tok) * a.q_stride + (int64_t)(r - tok * a.n_heads) * W;
    s_.limit = limit_of(rg * 16 + col);
#pragma unroll
    for (int k = 0; k < S::KS; ++k) s_.q[k] = load_frag8<T>(qr + 32 * k + 8 * grp);
  }
#pragma unroll
  for (int v = 0; v < S::RV; ++v) s_.my_limit[v] = limit_of(32 * v + (lane & 31));
  // (behind the last tile rows that do not exist are fetched)
  for (int tile = tile0; tile < tiles_end; tile += 2) {
    fetched();
    aim(tile + 1, x.have[1]);
    if (!s_.template step<SAFE>(even, x.have[0], weights, x, tile * KB, least, c, lane, wave,
                                [&](int b) { fetch(b, odd); }))
      return false;
    if (tile + 1 == tiles_end) break;
    fetched();
    aim(tile + 2, x.have[0]);
    if (!s_.template step<SAFE>(odd, x.have[1], weights, x, (tile + 1) * KB, least, c, lane, wave,
                                [&](int b) { fetch(b, even); }))
      return false;
  }
  fetched();

  // the sum of weights of each row, over lanes and waves
  {
    float y = s_.sum;
    y += __shfl_xor(y, 16);
    y += __shfl_xor(y, 32);
    int any = s_.seen;
    any |= __shfl_xor(any, 16);
    any |= __shfl_xor(any, 32);
    x.sums[kg][rg * 16 + col] = y;
    x.seen[kg][rg * 16 + col] = any;
  }
  __syncthreads();
  if (tile0 == 0 && wave == 0) {
    const int64_t id = g.cu ? first_block<R>(s.start, a.n_heads, n_now) : (int64_t)n_now * s.units;
    if (ws.by_unit || pc.more > 0)
      ws.heads[ws.by_unit ? id + unit : run] = int4{run, pc.more, s.start * a.n_heads + row0, min(n_rows - row0, R)};
  }
  const int tok0 = row0 / a.n_heads;
  const auto out = make_rsrc(static_cast<char*>(a.o) + (s.start + tok0) * a.o_stride * ES, INT32_MAX);
#pragma unroll
  for (int v = 0; v < S::RV; ++v) {
    const int r = 32 * v + (lane & 31);
    float all = 0.f;
    int some = 0;
#pragma unroll
    for (int k = 0; k < S::KG; ++k) all += x.sums[k][r], some |= x.seen[k][r];
    if (tile0 == 0 && tile1 == s.tiles - setup_of(S::KB)) {
      const int tok = (row0 + r) / a.n_heads;
      const int at = (int)((tok - tok0) * a.o_stride + (row0 + r - tok * a.n_heads) * DC + S::COLS * wave + 4 * h) * ES;
      const float inv = some ? __builtin_amdgcn_rcpf(all) : 0.f;  // no key: O is 0
#pragma unroll
      for (int d = 0; d < S::NV; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          typename Vec4<T>::type y;
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(s_.o[d][v][4 * b + e] * inv);
          store4(y, out, row0 + r < n_rows ? at + (32 * d + 8 * b) * ES : kBufferOff);
        }
    } else {
      const int64_t place = 2 * (int64_t)run + (tile0 == 0 ? 1 : 0);
      float* sums = ws.sums + (place * R + r) * DC + S::COLS * wave;
#pragma unroll
      for (int d = 0; d < S::NV; ++d)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<f32x4*>(sums + 32 * d + 8 * b + 4 * h) =
              f32x4{s_.o[d][v][4 * b], s_.o[d][v][4 * b + 1], s_.o[d][v][4 * b + 2], s_.o[d][v][4 * b + 3]};
      if (wave == 0) ws.stats[place * R + r] = float2{s_.top_o[v], some ? all : -1.f};
    }
  }
  end_of_variant<SAFE>();
  return true;
}

template <typename T, int DC, int DR, int R>
__global__ __launch_bounds__((Shape<T, DC, DR, R>::THREADS), 1) void latent_attend_kernel(LatentAttendArgs a, Workspace ws) {
  using S = Shape<T, DC, DR, R>;
  using A = Attend<T, DC, DR, R>;
  constexpr int KB = S::KB, THREADS = S::THREADS;
  __shared__ __attribute__((aligned(128))) char even[S::tile];
  __shared__ __attribute__((aligned(128))) char odd[S::tile];
  __shared__ __attribute__((aligned(16))) char weights[R * S::p_row];
  __shared__ typename A::Exchange x;
  __shared__ int64_t waves[S::NW], found[2];
  const LatentPages& g = a.pages;

  // this workgroup's run of tiles, and the sequence it begins in
  const int run = blockIdx.x;
  if (!ws.by_unit && threadIdx.x == 0) ws.heads[run].y = 0;
  // (a thread sums up the tiles of some neighbouring sequences, and the one that has the
  // run's first tile among its own looks for it there)
  const int each = (g.n_seqs - 1) / THREADS + 1, first = min((int)threadIdx.x * each, g.n_seqs);
  int64_t mine = 0, total;
  for (int i = first; i < min(first + each, g.n_seqs); ++i) mine += sequence_of<R, KB>(g, a.n_heads, i).all();
  const int64_t upto = scan<S::NW>(mine, waves, &total);
  const Runs<KB> runs(uniform(total), gridDim.x);
  if (run >= runs.runs) return;
  const int64_t lo = runs.begin(run), hi = runs.begin(run + 1);
  if (lo >= hi) return;
  if (mine > 0 && upto - mine <= lo && lo < upto) {
    int64_t at = upto - mine;
    int i = first;
    for (; i < first + each - 1 && i < g.n_seqs - 1; ++i) {
      const int64_t y = sequence_of<R, KB>(g, a.n_heads, i).all();
      if (lo < at + y) break;
      at += y;
    }
    found[0] = i;
    found[1] = at;
  }
  __syncthreads();
  int n = uniform((int)found[0]);
  int64_t seq_at = uniform(found[1]);  // the tile that the sequence's first unit begins with

  for (int64_t pos = lo; pos < hi;) {
    const Sequence s = sequence_of<R, KB>(g, a.n_heads, n);
    const int64_t in_seq = pos - seq_at;
    const int unit = (int)divide(in_seq, s.tiles), from = (int)(in_seq - (int64_t)unit * s.tiles);
    const int to = (int)min((int64_t)s.tiles, from + (hi - pos));
    pos += to - from;
    const Piece pc = {n, unit, max(from - setup_of(KB), 0), max(to - setup_of(KB), 0), run, runs.reached(run, s.tiles - to)};
    if (pos - seq_at >= s.all()) {
      seq_at = pos;
      ++n;
      while (n < g.n_seqs && sequence_of<R, KB>(g, a.n_heads, n).units == 0) ++n;
    }
    if (pc.tile1 > 0 && !attend_piece<T, DC, DR, R, false>(a, ws, s, pc, even, odd, weights, x))
      attend_piece<T, DC, DR, R, true>(a, ws, s, pc, even, odd, weights, x);
    if (n >= g.n_seqs) break;
  }
}

// The rows of units that were cut: the pieces' sums, each at its own maximum, brought
// to the largest.  A workgroup takes COLS columns of a row at a time, its threads in
// groups of COLS / 4 with every so many-th piece each; `shares` workgroups share a unit.
template <typename T, int DC, int R, int KB, int COLS>
__global__ __launch_bounds__(JOIN_THREADS) void latent_join_kernel(LatentAttendArgs a, Workspace ws, int shares) {
  constexpr int PARTS = DC / COLS, WIDTH = COLS / 4, GROUPS = JOIN_THREADS / WIDTH;
  __shared__ float factors[RUNS], wide[GROUPS][COLS];
  __shared__ float tops[4], sums[4];
  __shared__ int some_by[4];
  const LatentPages& g = a.pages;
  const int id = blockIdx.x / shares;
  if (ws.by_unit && g.cu) {  // a number may be no unit's, and its head then was not written
    const int n = find_sequence<R>(g.cu, g.n_seqs, g.t_total, a.n_heads, id);
    const Sequence s = sequence_of<R, KB>(g, a.n_heads, n);
    const int64_t unit = id - first_block<R>(s.start, a.n_heads, n);
    if (unit < 0 || unit >= s.units) return;
  }
  const int4 head = ws.heads[id];
  const int more = head.y;
  if (more == 0) return;
  const float c = a.scale * kLog2e;
  const int i = threadIdx.x, lane = i & 63, wave = i >> 6;
  const int group = i / WIDTH, at = 4 * (i % WIDTH);
  for (int item = blockIdx.x % shares; item < R * PARTS; item += shares) {
    const int part = item % PARTS, r = item / PARTS;
    if (r >= head.w) return;
    const auto place = [&](int k) { return ((int64_t)(k == 0 ? 2 * head.x + 1 : 2 * (head.x + k)) * R + r); };
    // a piece each thread: at most RUNS of them
    const float2 st = i <= more ? ws.stats[place(i)] : float2{0.f, -1.f};
    const bool mine = !(st.y == -1.f);
    float top = mine ? st.x : -__builtin_inff();
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    __syncthreads();
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    const float base = top == -__builtin_inff() ? 0.f : __fmul_rn(top, c);
    const float f = mine ? fast_exp2(__fmul_rn(st.x, c) - base) : 0.f;
    factors[i] = f;
    float sum = mine ? f * st.y : 0.f;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    const bool any = __any(mine);
    if (lane == 0) sums[wave] = sum, some_by[wave] = any;
    __syncthreads();
    f32x4 o = zero4();
#pragma unroll 4
    for (int k = group; k <= more; k += GROUPS)
      o += factors[k] * *reinterpret_cast<const f32x4*>(ws.sums + place(k) * DC + COLS * part + at);
    *reinterpret_cast<f32x4*>(&wide[group][at]) = o;
    __syncthreads();
    sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
    const float inv = some_by[0] | some_by[1] | some_by[2] | some_by[3] ? 1.f / sum : 0.f;
    const int row = head.z + r, tok = row / a.n_heads;
    T* out = static_cast<T*>(a.o) + (int64_t)tok * a.o_stride + (int64_t)(row - tok * a.n_heads) * DC + COLS * part;
    for (int col = i; col < COLS; col += JOIN_THREADS) {
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) y += wide[k][col];
      out[col] = from_f32<T>(y * inv);
    }
  }
}

template <typename T, int DC, int DR, int R>
hipError_t run(const LatentAttendArgs& a, const Plan& plan, const Workspace& ws, hipStream_t stream) {
  hipError_t e = enqueue(latent_attend_kernel<T, DC, DR, R>, (unsigned)plan.runs, Shape<T, DC, DR, R>::THREADS, stream, a, ws);
  if (e != hipSuccess || plan.runs == 1) return e;  // (a single run cuts no unit)
  constexpr int KB = Shape<T, DC, DR, R>::KB;
  if (plan.units <= FEW_UNITS / 8)  // their rows alone would not fill the GPU
    return enqueue(latent_join_kernel<T, DC, R, KB, 128>, (unsigned)(plan.heads * R * (DC / 128)), JOIN_THREADS, stream, a,
                   ws, R * (DC / 128));
  const int shares = plan.by_unit ? R : JOIN_SHARES;
  return enqueue(latent_join_kernel<T, DC, R, KB, DC>, (unsigned)(plan.heads * shares), JOIN_THREADS, stream, a, ws, shares);
}

template <typename T, int R>
hipError_t by_shape(const LatentAttendArgs& a, const Plan& plan, const Workspace& ws, hipStream_t stream) {
  if (a.dc == 512)
    return a.dr == 64 ? run<T, 512, 64, R>(a, plan, ws, stream) : run<T, 512, 32, R>(a, plan, ws, stream);
  return a.dr == 64 ? run<T, 256, 64, R>(a, plan, ws, stream) : run<T, 256, 32, R>(a, plan, ws, stream);
}

}  // namespace

size_t latent_workspace_bytes(const LatentAttendArgs& a) {
  return a.pages.t_total == 0 || a.pages.n_seqs == 0 ? 0 : Plan(a).bytes;
}

hipError_t launch_latent_attend(const LatentAttendArgs& a, void* workspace, hipStream_t stream) {
  if (a.pages.t_total == 0 || a.pages.n_seqs == 0) return hipSuccess;
  const Plan plan(a);
  char* w = static_cast<char*>(workspace);
  const Workspace ws = {reinterpret_cast<int4*>(w), reinterpret_cast<float*>(w + plan.heads_bytes),
                        reinterpret_cast<float2*>(w + plan.heads_bytes + plan.sums_bytes), plan.by_unit};
  if (!a.bf16) return by_shape<float, 32>(a, plan, ws, stream);
  return plan.rows == 64 ? by_shape<bf16, 64>(a, plan, ws, stream) : by_shape<bf16, 32>(a, plan, ws, stream);
}

}  // namespace kda
