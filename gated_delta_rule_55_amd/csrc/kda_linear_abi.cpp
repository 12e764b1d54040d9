// kda_linear_abi.cpp -- the C ABI declared in include/kda_linear.h: descriptor
// validation on the host, then launches on the caller's stream.  Every check
// runs before anything is enqueued.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kda_check.h"
#include "kda_linear.h"
#include "kda_linear_launch.h"

namespace {

using kda::aligned;
using kda::overlap;
using kda::Range;
using kda::range_of;
using kda::row_set;
using kda::RowSet;

// Workgroups of a launch: 256 threads each stay below 2^32.
constexpr int64_t kMaxBlocks = (int64_t)1 << 24;
constexpr int64_t kMaxStride = (int64_t)1 << 22;
// (slot, head) states of a pool: keeps its size in bytes in 64 bits.
constexpr int64_t kMaxStates = (int64_t)1 << 40;

int check_heads(int32_t n_heads, int32_t n_k_heads, int32_t dk, int32_t dv, int* kheads) {
  if (n_heads < 1 || n_heads > 65535) return KDA_ERR_SHAPE;
  const int hk = n_k_heads == 0 ? n_heads : n_k_heads;
  if (hk < 1 || hk > n_heads || n_heads % hk != 0) return KDA_ERR_SHAPE;
  if (!kda::supported_d(dk) || !kda::supported_d(dv)) return KDA_ERR_UNSUPPORTED;
  *kheads = hk;
  return KDA_OK;
}

// A token stride in elements: 0 = dense; else at least the row, a multiple of
// 16 bytes, and at most 2^22, which keeps the byte offsets of a 64-token chunk
// in 31 bits.
int check_stride(int64_t stride, int64_t row, int64_t es, int64_t* out) {
  if (stride != 0 && (stride < row || stride * es % 16 != 0 || stride > kMaxStride))
    return KDA_ERR_SHAPE;
  *out = stride == 0 ? row : stride;
  return *out <= kMaxStride ? KDA_OK : KDA_ERR_SHAPE;
}

int check_linear(const kda_linear_prefill_desc* d, kda::LinearPrefillArgs* a) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_linear_prefill_desc)) return KDA_ERR_VERSION;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (d->n_seqs < 1 || d->t_total < 0 || d->t_total > INT32_MAX - 64) return KDA_ERR_SHAPE;
  int st = check_heads(d->n_heads, d->n_k_heads, d->dk, d->dv, &a->kheads);
  if (st != KDA_OK) return st;
  if (d->decay != KDA_DECAY_TOKEN && d->decay != KDA_DECAY_HEAD) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(d->scale)) return KDA_ERR_SHAPE;
  if (d->state_indices && (d->n_slots < 1 || (int64_t)d->n_slots * d->n_heads > kMaxStates))
    return KDA_ERR_SHAPE;
  st = kda::check_state_dtype(d->state_dtype, d->dtype, &a->state_bf16);
  if (st != KDA_OK) return st;
  a->bf16 = d->dtype == KDA_DTYPE_BF16;
  const int64_t es = a->bf16 ? 2 : 4, H = d->n_heads;
  if ((st = check_stride(d->q_stride, (int64_t)a->kheads * d->dk, es, &a->q_stride)) != KDA_OK ||
      (st = check_stride(d->k_stride, (int64_t)a->kheads * d->dk, es, &a->k_stride)) != KDA_OK ||
      (st = check_stride(d->v_stride, H * d->dv, es, &a->v_stride)) != KDA_OK ||
      (st = check_stride(d->o_stride, H * d->dv, es, &a->o_stride)) != KDA_OK)
    return st;
  a->decay_head = d->decay == KDA_DECAY_HEAD;
  a->n_seqs = d->n_seqs;
  a->n_heads = d->n_heads;
  a->dk = d->dk;
  a->dv = d->dv;
  a->t_total = d->t_total;
  a->scale = d->scale != 0.f ? d->scale : 1.0f / std::sqrt((float)d->dk);
  // the kernels hold a segment's length in 32 bits
  const int64_t seg = kda::linear_segment(a->t_total, a->n_seqs, a->n_heads, a->dv, a->bf16);
  if (seg > INT32_MAX) return KDA_ERR_SHAPE;
  // workgroups: segments x heads, and 8 per segment length and head that join them
  if ((kda::linear_segments(a->t_total, a->n_seqs, seg) + 8) * H >= kMaxBlocks ||
      a->t_total / seg * H * 8 >= kMaxBlocks)
    return KDA_ERR_SHAPE;
  return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_linear_workspace_bytes(const kda_linear_prefill_desc* d, int* status) {
  kda::LinearPrefillArgs a{};
  const int st = check_linear(d, &a);
  if (status) *status = st;
  return st == KDA_OK ? kda::linear_workspace_bytes(a) : 0;
}

int kda_linear_prefill(const kda_linear_prefill_desc* d, void* workspace, size_t workspace_bytes,
                       void* stream) {
  kda::LinearPrefillArgs a{};
  const int st = check_linear(d, &a);
  if (st != KDA_OK) return st;
  const int64_t T = d->t_total, H = d->n_heads, N = d->n_seqs;
  if (!d->cu_seqlens && N != 1) return KDA_ERR_NULL;
  if (T > 0 && (!d->q || !d->k || !d->v || !d->g || !d->o)) return KDA_ERR_NULL;
  const void* p16[] = {d->q, d->k, d->v, d->o, d->h0, d->ht};
  for (const void* p : p16)
    if (p && !aligned(p, 16)) return KDA_ERR_ALIGN;
  const void* p4[] = {d->g, d->cu_seqlens, d->state_indices};
  for (const void* p : p4)
    if (p && !aligned(p, 4)) return KDA_ERR_ALIGN;
  const size_t need = kda::linear_workspace_bytes(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return KDA_ERR_ALIGN;

  const int64_t es = a.bf16 ? 2 : 4, ess = a.state_bf16 ? 2 : 4;
  const int64_t states = (d->state_indices ? (int64_t)d->n_slots : N) * H * d->dk * d->dv * ess;
  const Range rh0 = range_of(d->h0, d->h0 ? states : 0), rht = range_of(d->ht, d->ht ? states : 0);
  const RowSet o = row_set(d->o, T, a.o_stride, H * d->dv, es);
  const RowSet qkv[] = {row_set(d->q, T, a.q_stride, (int64_t)a.kheads * d->dk, es),
                        row_set(d->k, T, a.k_stride, (int64_t)a.kheads * d->dk, es),
                        row_set(d->v, T, a.v_stride, H * d->dv, es)};
  const Range ro = range_of(o), rw = range_of(workspace, (int64_t)need);
  for (const RowSet& r : qkv)
    if (overlap(o, r) || overlap(rht, range_of(r)) || overlap(rw, range_of(r))) return KDA_ERR_ALIAS;
  const Range ins[] = {
      range_of(d->g, d->g ? (a.decay_head ? H : T * H) * 4 : 0),
      range_of(d->cu_seqlens, d->cu_seqlens ? (N + 1) * 4 : 0),
      range_of(d->state_indices, d->state_indices ? N * 4 : 0)};
  for (const Range& r : ins)
    if (overlap(ro, r) || overlap(rht, r) || overlap(rw, r)) return KDA_ERR_ALIAS;
  // ht may be exactly h0 (in-place carry) but may not partly overlap it
  if (overlap(ro, rh0) || overlap(ro, rht) || (d->ht != d->h0 && overlap(rht, rh0)))
    return KDA_ERR_ALIAS;
  if (overlap(rw, ro) || overlap(rw, rh0) || overlap(rw, rht)) return KDA_ERR_ALIAS;

  a.q = d->q;
  a.k = d->k;
  a.v = d->v;
  a.g = d->g;
  a.o = d->o;
  a.h0 = d->h0;
  a.ht = d->ht;
  a.cu_seqlens = d->cu_seqlens;
  a.slots = d->state_indices;
  a.n_slots = d->state_indices ? d->n_slots : 0;
  return kda::hip_status(kda::launch_linear_prefill(a, workspace, (hipStream_t)stream));
}

int kda_linear_decode(const kda_linear_decode_desc* d, void* stream) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_linear_decode_desc)) return KDA_ERR_VERSION;
  if (d->dtype != KDA_DTYPE_F32 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (d->n_seqs < 0) return KDA_ERR_SHAPE;
  kda::LinearDecodeArgs a{};
  int st = check_heads(d->n_heads, d->n_k_heads, d->dk, d->dv, &a.kheads);
  if (st != KDA_OK) return st;
  if (d->decay != KDA_DECAY_TOKEN && d->decay != KDA_DECAY_HEAD) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(d->scale)) return KDA_ERR_SHAPE;
  if (d->state_indices && (d->n_slots < 1 || (int64_t)d->n_slots * d->n_heads > kMaxStates))
    return KDA_ERR_SHAPE;
  st = kda::check_state_dtype(d->state_dtype, d->dtype, &a.state_bf16);
  if (st != KDA_OK) return st;
  a.bf16 = d->dtype == KDA_DTYPE_BF16;
  const int64_t es = a.bf16 ? 2 : 4, ess = a.state_bf16 ? 2 : 4, H = d->n_heads, N = d->n_seqs;
  if ((st = check_stride(d->q_stride, (int64_t)a.kheads * d->dk, es, &a.q_stride)) != KDA_OK ||
      (st = check_stride(d->k_stride, (int64_t)a.kheads * d->dk, es, &a.k_stride)) != KDA_OK ||
      (st = check_stride(d->v_stride, H * d->dv, es, &a.v_stride)) != KDA_OK ||
      (st = check_stride(d->o_stride, H * d->dv, es, &a.o_stride)) != KDA_OK)
    return st;
  if (N * H >= kMaxBlocks) return KDA_ERR_SHAPE;
  if (N == 0) return KDA_OK;
  if (!d->state || !d->q || !d->k || !d->v || !d->g || !d->o) return KDA_ERR_NULL;
  const void* p16[] = {d->state, d->q, d->k, d->v, d->o};
  for (const void* p : p16)
    if (!aligned(p, 16)) return KDA_ERR_ALIGN;
  if (!aligned(d->g, 4) || (d->state_indices && !aligned(d->state_indices, 4))) return KDA_ERR_ALIGN;
  const Range rs = range_of(d->state, (d->state_indices ? (int64_t)d->n_slots : N) * H * d->dk *
                                          d->dv * ess);
  const RowSet o = row_set(d->o, N, a.o_stride, H * d->dv, es);
  const RowSet qkv[] = {row_set(d->q, N, a.q_stride, (int64_t)a.kheads * d->dk, es),
                        row_set(d->k, N, a.k_stride, (int64_t)a.kheads * d->dk, es),
                        row_set(d->v, N, a.v_stride, H * d->dv, es)};
  const Range ro = range_of(o);
  for (const RowSet& r : qkv)
    if (overlap(o, r) || overlap(rs, range_of(r))) return KDA_ERR_ALIAS;
  const Range ins[] = {
      range_of(d->g, (d->decay == KDA_DECAY_HEAD ? H : N * H) * 4),
      range_of(d->state_indices, d->state_indices ? N * 4 : 0)};
  for (const Range& r : ins)
    if (overlap(ro, r) || overlap(rs, r)) return KDA_ERR_ALIAS;
  if (overlap(ro, rs)) return KDA_ERR_ALIAS;
  a.decay_head = d->decay == KDA_DECAY_HEAD;
  a.n_seqs = d->n_seqs;
  a.n_heads = d->n_heads;
  a.dk = d->dk;
  a.dv = d->dv;
  a.scale = d->scale != 0.f ? d->scale : 1.0f / std::sqrt((float)d->dk);
  a.state = d->state;
  a.q = d->q;
  a.k = d->k;
  a.v = d->v;
  a.g = d->g;
  a.o = d->o;
  a.slots = d->state_indices;
  a.n_slots = d->state_indices ? d->n_slots : 0;
  return kda::hip_status(kda::launch_linear_decode(a, (hipStream_t)stream));
}

}  // extern "C"
