// kda_latent_abi.cpp -- the C ABI declared in include/kda_latent.h: descriptor
// validation on the host, then launches on the caller's stream.  Every check
// runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "kda_check.h"
#include "kda_latent.h"
#include "kda_latent_launch.h"

namespace {

using kda::aligned;
using kda::overlap;
using kda::Range;
using kda::range_of;
using kda::row_set;
using kda::RowSet;

constexpr int64_t kMaxStride = (int64_t)1 << 28;
// Of rows that a workgroup addresses from its first one: keeps the byte offsets of 128 of
// them in 31 bits.
constexpr int64_t kMaxRowStride = (int64_t)1 << 22;
constexpr int64_t kMaxSequences = (int64_t)1 << 24;
// A kernel counts positions some tiles past the last one.
constexpr int64_t kMaxPositions = INT32_MAX - 256;
constexpr int64_t kMaxTokens = INT32_MAX - 64;
// Workgroups of a launch: threads stay below 2^32.
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;

bool dtype_ok(int32_t dtype) { return dtype == KDA_DTYPE_F32 || dtype == KDA_DTYPE_BF16; }
bool heads_ok(int32_t n) { return n >= 1 && n <= 65535; }
bool tokens_ok(int64_t n) { return n >= 0 && n <= kMaxTokens; }
// A scale that fp32 holds as a normal number, times log2(e) too.
bool scale_ok(float s) { return std::isfinite(1.5f * s) && s >= FLT_MIN; }

// A stride in elements: 0 = dense; else at least `row`, a multiple of 16 bytes and at
// most 2^28.
int check_stride(int64_t stride, int64_t row, int64_t es, int64_t* out) {
  if (stride != 0 && (stride < row || stride * es % 16 != 0 || stride > kMaxStride)) return KDA_ERR_SHAPE;
  *out = stride == 0 ? row : stride;
  return *out <= kMaxStride ? KDA_OK : KDA_ERR_SHAPE;
}

// Strides of [rows, H, d]: heads within a row, rows past the last head's end.
int check_head_strides(int64_t stride, int64_t head_stride, int64_t heads, int64_t d, int64_t es, int64_t* out,
                       int64_t* head_out) {
  int st = check_stride(head_stride, d, es, head_out);
  if (st != KDA_OK) return st;
  const int64_t row = (heads - 1) * *head_out + d;
  if (stride == 0) {
    *out = heads * *head_out;
    return *out <= kMaxStride ? KDA_OK : KDA_ERR_SHAPE;
  }
  return check_stride(stride, row, es, out);
}

// [rows, heads, d] as rows of d at the head stride where these are at one stride, else
// (conservatively) as rows from the first head's start to the last one's end.
RowSet head_rows(const void* p, int64_t rows, int64_t stride, int64_t heads, int64_t head_stride, int64_t d, int64_t es) {
  if (heads * head_stride == stride) return row_set(p, rows * heads, head_stride, d, es);
  return row_set(p, rows, stride, (heads - 1) * head_stride + d, es);
}

// Whether two sets of heads at the same strides share a byte: rows r apart and heads k apart do
// where |by - r stride - k head| < d.  A row ends before the next begins, and a head too, so two
// values of each can.  (Bytes.)
bool heads_overlap(const void* x, const void* y, int64_t rows, int64_t stride, int64_t heads, int64_t head, int64_t d) {
  const int64_t by = (int64_t)((uintptr_t)y - (uintptr_t)x);
  const auto below = [](int64_t a, int64_t b) { return a / b - (a % b < 0 ? 1 : 0); };
  for (int64_t r = below(by, stride), i = 0; i < 2; ++i, ++r) {
    if (r <= -rows || r >= rows) continue;
    const int64_t rest = by - r * stride;
    for (int64_t k = below(rest, head), j = 0; j < 2; ++j, ++k)
      if (k > -heads && k < heads && rest - k * head < d && k * head - rest < d) return true;
  }
  return false;
}

int check_pages(int32_t dtype, int32_t n_seqs, int32_t dc, int32_t dr, int32_t page_size, int32_t max_pages,
                int32_t n_pages, int64_t page_stride, int64_t row_stride, int64_t t_total, bool cu, kda::LatentPages* g) {
  if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
  if (n_seqs < 0 || n_seqs > kMaxSequences || page_size < 1 || max_pages < 1 || n_pages < 0 || !tokens_ok(t_total) ||
      (int64_t)max_pages * page_size > kMaxPositions || (!cu && t_total != n_seqs))
    return KDA_ERR_SHAPE;
  if ((dc != 256 && dc != 512) || (dr != 32 && dr != 64)) return KDA_ERR_UNSUPPORTED;
  const int64_t es = dtype == KDA_DTYPE_BF16 ? 2 : 4;
  int st = check_stride(row_stride, dc + dr, es, &g->row_stride);
  if (st != KDA_OK) return st;
  const int64_t page = ((int64_t)page_size - 1) * g->row_stride + dc + dr;
  if (page_stride == 0) {
    g->page_stride = page_size * g->row_stride;
  } else {
    if (page_stride < page || page_stride * es % 16 != 0) return KDA_ERR_SHAPE;
    g->page_stride = page_stride;
  }
  // keeps the pool's size in bytes in 64 bits
  if (g->page_stride > ((int64_t)1 << 40)) return KDA_ERR_SHAPE;
  if (n_pages > 0 && g->page_stride > ((int64_t)1 << 60) / n_pages) return KDA_ERR_SHAPE;
  g->page_size = page_size;
  g->page_shift = 31;
  while (((int64_t)1 << (g->page_shift - 31)) < page_size) ++g->page_shift;
  g->page_factor = (uint32_t)((((uint64_t)1 << g->page_shift) + page_size - 1) / page_size);
  g->max_pages = max_pages;
  g->n_pages = n_pages;
  g->n_seqs = n_seqs;
  g->t_total = (int)t_total;
  return KDA_OK;
}

Range cache_range(const void* p, const kda::LatentPages& g, int64_t w, int64_t es) {
  if (!p || g.n_pages == 0) return range_of(p, 0);
  return range_of(p, ((g.n_pages - 1) * g.page_stride + (g.page_size - 1) * g.row_stride + w) * es);
}

int check_tables(const int32_t* table, const int32_t* lens, const int32_t* cu, const kda::LatentPages& g, Range (&r)[3]) {
  if (!table || !lens) return KDA_ERR_NULL;
  if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(cu, 4)) return KDA_ERR_ALIGN;
  r[0] = range_of(table, (int64_t)g.n_seqs * g.max_pages * 4);
  r[1] = range_of(lens, (int64_t)g.n_seqs * 4);
  r[2] = range_of(cu, cu ? ((int64_t)g.n_seqs + 1) * 4 : 0);
  return KDA_OK;
}

int check_attend(const kda_latent_attend_desc* d, kda::LatentAttendArgs* a) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_latent_attend_desc)) return KDA_ERR_VERSION;
  int st = check_pages(d->dtype, d->n_seqs, d->dc, d->dr, d->page_size, d->max_pages, d->n_pages, d->page_stride,
                       d->row_stride, d->t_total, d->cu_seqlens != nullptr, &a->pages);
  if (st != KDA_OK) return st;
  if (!heads_ok(d->n_heads) || !scale_ok(d->scale)) return KDA_ERR_SHAPE;
  const int64_t es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4, H = d->n_heads;
  if ((st = check_stride(d->q_stride, H * (d->dc + d->dr), es, &a->q_stride)) != KDA_OK ||
      (st = check_stride(d->o_stride, H * d->dc, es, &a->o_stride)) != KDA_OK)
    return st;
  // (token, head) rows are counted in 32 bits
  if (a->o_stride > kMaxRowStride || d->t_total * H > kMaxTokens)
    return KDA_ERR_SHAPE;
  a->bf16 = d->dtype == KDA_DTYPE_BF16;
  a->n_heads = d->n_heads;
  a->dc = d->dc;
  a->dr = d->dr;
  a->scale = d->scale;
  a->pages.cu = d->cu_seqlens;
  return KDA_OK;
}

// What depends on sizes alone.
int check_prefill(const kda_latent_prefill_desc* d, kda::LatentPrefillArgs* a) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_latent_prefill_desc)) return KDA_ERR_VERSION;
  if (!dtype_ok(d->dtype)) return KDA_ERR_DTYPE;
  if (d->n_seqs < 1 || !heads_ok(d->n_heads) || !tokens_ok(d->q_total) || !tokens_ok(d->k_total)) return KDA_ERR_SHAPE;
  if ((d->dn != 64 && d->dn != 128) || (d->dv != 64 && d->dv != 128) || (d->dr != 32 && d->dr != 64))
    return KDA_ERR_UNSUPPORTED;
  if (d->scale != 0.f && !scale_ok(d->scale)) return KDA_ERR_SHAPE;
  const int64_t T = d->q_total, K = d->k_total, H = d->n_heads, N = d->n_seqs;
  const int64_t dn = d->dn, dr = d->dr, dv = d->dv, es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  if (kda::latent_query_blocks(T, N) * H >= kMaxBlocks || (!d->cu_seqlens_k && K != T)) return KDA_ERR_SHAPE;
  int st;
  if ((st = check_stride(d->q_stride, H * (dn + dr), es, &a->q_stride)) != KDA_OK ||
      (st = check_head_strides(d->k_stride, d->k_head_stride, H, dn, es, &a->k_stride, &a->k_head)) != KDA_OK ||
      (st = check_stride(d->k_pe_stride, dr, es, &a->pe_stride)) != KDA_OK ||
      (st = check_head_strides(d->v_stride, d->v_head_stride, H, dv, es, &a->v_stride, &a->v_head)) != KDA_OK ||
      (st = check_stride(d->o_stride, H * dv, es, &a->o_stride)) != KDA_OK)
    return st;
  if (a->k_stride > kMaxRowStride || a->pe_stride > kMaxRowStride || a->v_stride > kMaxRowStride ||
      a->o_stride > kMaxRowStride)
    return KDA_ERR_SHAPE;
  a->bf16 = d->dtype == KDA_DTYPE_BF16;
  a->n_seqs = d->n_seqs;
  a->n_heads = d->n_heads;
  a->dn = d->dn;
  a->dr = d->dr;
  a->dv = d->dv;
  a->q_total = (int)T;
  a->k_total = (int)K;
  a->scale = d->scale != 0.f ? d->scale : 1.0f / std::sqrt((float)(dn + dr));
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_latent_prefill_workspace_bytes(const kda_latent_prefill_desc* d, int* status) {
  kda::LatentPrefillArgs a{};
  const int st = check_prefill(d, &a);
  if (status) *status = st;
  return st == KDA_OK ? kda::latent_prefill_workspace_bytes(a) : 0;
}

int kda_latent_prefill(const kda_latent_prefill_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
  kda::LatentPrefillArgs a{};
  const int st = check_prefill(d, &a);
  if (st != KDA_OK) return st;
  const int64_t T = d->q_total, K = d->k_total, H = d->n_heads, N = d->n_seqs;
  const int64_t dn = d->dn, dr = d->dr, dv = d->dv, es = a.bf16 ? 2 : 4;
  if ((!d->cu_seqlens || (d->cu_seqlens_k && !d->cu_seqlens)) && N != 1) return KDA_ERR_NULL;
  if (T > 0 && (!d->q || !d->o)) return KDA_ERR_NULL;
  if (T > 0 && K > 0 && (!d->k || !d->k_pe || !d->v)) return KDA_ERR_NULL;
  const void* p16[] = {d->q, d->k, d->k_pe, d->v, d->o};
  for (const void* p : p16)
    if (!aligned(p, 16)) return KDA_ERR_ALIGN;
  if (!aligned(d->cu_seqlens, 4) || !aligned(d->cu_seqlens_k, 4)) return KDA_ERR_ALIGN;
  const size_t need = kda::latent_prefill_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return KDA_ERR_ALIGN;
  const Range rw = range_of(workspace, (int64_t)need);
  const RowSet o = row_set(d->o, T, a.o_stride, H * dv, es);
  const RowSet ins[] = {row_set(d->q, T, a.q_stride, H * (dn + dr), es),
                        head_rows(d->k, K, a.k_stride, H, a.k_head, dn, es), row_set(d->k_pe, K, a.pe_stride, dr, es),
                        head_rows(d->v, K, a.v_stride, H, a.v_head, dv, es)};
  for (const RowSet& r : ins)
    if (overlap(o, r) || overlap(rw, range_of(r))) return KDA_ERR_ALIAS;
  const Range tables[] = {range_of(d->cu_seqlens, d->cu_seqlens ? (N + 1) * 4 : 0),
                          range_of(d->cu_seqlens_k, d->cu_seqlens_k ? (N + 1) * 4 : 0)};
  for (const Range& r : tables)
    if (overlap(range_of(o), r) || overlap(rw, r)) return KDA_ERR_ALIAS;
  if (overlap(rw, range_of(o))) return KDA_ERR_ALIAS;
  a.q = d->q;
  a.k = d->k;
  a.pe = d->k_pe;
  a.v = d->v;
  a.o = d->o;
  a.cu = d->cu_seqlens;
  a.cu_k = d->cu_seqlens_k;
  return kda::hip_status(kda::launch_latent_prefill(a, workspace, (hipStream_t)stream));
}

size_t kda_latent_workspace_bytes(const kda_latent_attend_desc* d, int* status) {
  kda::LatentAttendArgs a{};
  const int st = check_attend(d, &a);
  if (status) *status = st;
  return st == KDA_OK ? kda::latent_workspace_bytes(a) : 0;
}

int kda_latent_attend(const kda_latent_attend_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
  kda::LatentAttendArgs a{};
  int st = check_attend(d, &a);
  if (st != KDA_OK) return st;
  kda::LatentPages& g = a.pages;
  if (d->n_seqs == 0 || d->t_total == 0) return KDA_OK;
  if (!d->q || !d->o || (d->n_pages > 0 && !d->cache)) return KDA_ERR_NULL;
  const void* p16[] = {d->q, d->o, d->cache};
  for (const void* p : p16)
    if (!aligned(p, 16)) return KDA_ERR_ALIGN;
  const int64_t es = a.bf16 ? 2 : 4, H = a.n_heads, W = a.dc + a.dr, T = d->t_total;
  Range in[5];
  Range tables[3];
  if ((st = check_tables(d->block_table, d->seq_lens, d->cu_seqlens, g, tables)) != KDA_OK) return st;
  const size_t need = kda::latent_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return KDA_ERR_ALIGN;
  const RowSet o = row_set(d->o, T, a.o_stride, H * a.dc, es), q = row_set(d->q, T, a.q_stride, H * W, es);
  if (overlap(o, q)) return KDA_ERR_ALIAS;
  const Range ro = range_of(o), rw = range_of(workspace, (int64_t)need);
  in[0] = tables[0], in[1] = tables[1], in[2] = tables[2], in[3] = cache_range(d->cache, g, W, es), in[4] = range_of(q);
  for (int i = 0; i < 5; ++i)
    if ((i < 4 && overlap(ro, in[i])) || overlap(rw, in[i])) return KDA_ERR_ALIAS;
  if (overlap(rw, ro)) return KDA_ERR_ALIAS;
  a.q = d->q;
  a.cache = d->cache;
  a.o = d->o;
  g.table = d->block_table;
  g.lens = d->seq_lens;
  return kda::hip_status(kda::launch_latent_attend(a, workspace, (hipStream_t)stream));
}

int kda_latent_append(const kda_latent_append_desc* d, void* stream) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_latent_append_desc)) return KDA_ERR_VERSION;
  kda::LatentAppendArgs a{};
  kda::LatentPages& g = a.pages;
  int st = check_pages(d->dtype, d->n_seqs, d->dc, d->dr, d->page_size, d->max_pages, d->n_pages, d->page_stride,
                       d->row_stride, d->t_total, d->cu_seqlens != nullptr, &g);
  if (st != KDA_OK) return st;
  if (d->t_total / 4 >= kMaxBlocks) return KDA_ERR_SHAPE;  // a workgroup for 4 tokens
  if (d->rotary != KDA_ROTARY_HALF && d->rotary != KDA_ROTARY_INTERLEAVED) return KDA_ERR_UNSUPPORTED;
  if (!(std::isfinite(d->eps) && d->eps >= 0.f) || !std::isfinite(d->magnitude)) return KDA_ERR_SHAPE;
  const int64_t es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4, W = d->dc + d->dr, T = d->t_total;
  if ((st = check_stride(d->latent_stride, d->dc, es, &a.latent_stride)) != KDA_OK ||
      (st = check_stride(d->k_pe_stride, d->dr, es, &a.pe_stride)) != KDA_OK ||
      (st = check_stride(d->rows_out_stride, W, es, &a.rows_stride)) != KDA_OK)
    return st;
  if (d->n_seqs == 0 || T == 0) return KDA_OK;
  if (!d->latent || !d->k_pe || (d->n_pages > 0 && !d->cache)) return KDA_ERR_NULL;
  const void* p16[] = {d->latent, d->k_pe, d->cache, d->rows_out};
  for (const void* p : p16)
    if (!aligned(p, 16)) return KDA_ERR_ALIGN;
  if (!aligned(d->weight, 4) || !aligned(d->frequencies, 8)) return KDA_ERR_ALIGN;
  Range tables[3];
  if ((st = check_tables(d->block_table, d->seq_lens, d->cu_seqlens, g, tables)) != KDA_OK) return st;
  const RowSet lat = row_set(d->latent, T, a.latent_stride, d->dc, es), pe = row_set(d->k_pe, T, a.pe_stride, d->dr, es);
  const RowSet out = row_set(d->rows_out, T, a.rows_stride, W, es);
  const Range cache = cache_range(d->cache, g, W, es);
  // rows_out may be where both inputs are, row for row (a single row has no stride: callers
  // give any)
  const bool in_place = d->rows_out && d->rows_out == d->latent &&
                        (const char*)d->k_pe == (const char*)d->latent + d->dc * es &&
                        (T == 1 || (a.rows_stride == a.latent_stride && a.rows_stride == a.pe_stride));
  if (!in_place && (overlap(out, lat) || overlap(out, pe))) return KDA_ERR_ALIAS;
  if (overlap(cache, range_of(lat)) || overlap(cache, range_of(pe)) || overlap(cache, range_of(out))) return KDA_ERR_ALIAS;
  const Range small[] = {tables[0], tables[1], tables[2], range_of(d->weight, d->weight ? (int64_t)d->dc * 4 : 0),
                         range_of(d->frequencies, d->frequencies ? (int64_t)d->dr * 4 : 0)};
  for (const Range& r : small)
    if (overlap(cache, r) || overlap(range_of(out), r)) return KDA_ERR_ALIAS;
  a.bf16 = d->dtype == KDA_DTYPE_BF16;
  a.dc = d->dc;
  a.dr = d->dr;
  a.interleaved = d->rotary == KDA_ROTARY_INTERLEAVED;
  a.eps = d->eps;
  a.magnitude = d->magnitude != 0.f ? d->magnitude : 1.f;
  a.latent = d->latent;
  a.pe = d->k_pe;
  a.cache = d->cache;
  a.rows = d->rows_out;
  a.weight = d->weight;
  a.frequencies = d->frequencies;
  g.table = d->block_table;
  g.lens = d->seq_lens;
  g.cu = d->cu_seqlens;
  return kda::hip_status(kda::launch_latent_append(a, (hipStream_t)stream));
}

int kda_rotary(const kda_rotary_desc* d, void* stream) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_rotary_desc)) return KDA_ERR_VERSION;
  if (!dtype_ok(d->dtype)) return KDA_ERR_DTYPE;
  if (!heads_ok(d->n_heads) || !tokens_ok(d->t_total) || !std::isfinite(d->magnitude)) return KDA_ERR_SHAPE;
  if (d->dim < 16 || d->dim > 256 || d->dim % 16 != 0) return KDA_ERR_UNSUPPORTED;
  if (d->rotary != KDA_ROTARY_HALF && d->rotary != KDA_ROTARY_INTERLEAVED) return KDA_ERR_UNSUPPORTED;
  kda::RotaryArgs a{};
  const int64_t es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4, T = d->t_total, H = d->n_heads;
  int st;
  if ((st = check_head_strides(d->x_stride, d->x_head_stride, H, d->dim, es, &a.x_stride, &a.x_head)) != KDA_OK ||
      (st = check_head_strides(d->y_stride, d->y_head_stride, H, d->dim, es, &a.y_stride, &a.y_head)) != KDA_OK)
    return st;
  // a workgroup for 256 / (8 x at most 64) tokens
  if (T * (H < 8 ? H : 8) * (d->dim / 4) / 256 >= kMaxBlocks) return KDA_ERR_SHAPE;
  if (T == 0) return KDA_OK;
  if (!d->x || !d->y || !d->positions || !d->frequencies) return KDA_ERR_NULL;
  if (!aligned(d->x, 16) || !aligned(d->y, 16) || !aligned(d->positions, 4) || !aligned(d->frequencies, 8))
    return KDA_ERR_ALIGN;
  const RowSet x = head_rows(d->x, T, a.x_stride, H, a.x_head, d->dim, es);
  const RowSet y = head_rows(d->y, T, a.y_stride, H, a.y_head, d->dim, es);
  // (a single row or head has no stride)
  const bool alike = (T == 1 || a.x_stride == a.y_stride) && (H == 1 || a.x_head == a.y_head);
  const bool in_place = d->x == d->y && alike;
  if (!in_place && overlap(x, y) &&
      (!alike || heads_overlap(d->x, d->y, T, a.x_stride * es, H, a.x_head * es, d->dim * es)))
    return KDA_ERR_ALIAS;
  if (overlap(range_of(y), range_of(d->positions, T * 4)) ||
      overlap(range_of(y), range_of(d->frequencies, (int64_t)d->dim * 4)))
    return KDA_ERR_ALIAS;
  a.bf16 = d->dtype == KDA_DTYPE_BF16;
  a.n_heads = d->n_heads;
  a.dim = d->dim;
  a.interleaved = d->rotary == KDA_ROTARY_INTERLEAVED;
  a.magnitude = d->magnitude != 0.f ? d->magnitude : 1.f;
  a.t_total = (int)T;
  a.x = d->x;
  a.y = d->y;
  a.positions = d->positions;
  a.frequencies = d->frequencies;
  return kda::hip_status(kda::launch_rotary(a, (hipStream_t)stream));
}

}  // extern "C"
