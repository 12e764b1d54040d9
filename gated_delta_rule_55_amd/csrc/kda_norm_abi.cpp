// kda_norm_abi.cpp -- the C ABI declared in include/kda_norm.h: descriptor
// validation on the host, then launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "kda_check.h"
#include "kda_norm.h"
#include "kda_norm_launch.h"

namespace {

using kda::aligned;
using kda::overlap;
using kda::Range;
using kda::range_of;

constexpr int kMaxDim = 16384;

struct Rows {
  const void* p;
  int64_t stride;  // resolved, elements
  int64_t es;
  kda::RowSet set;
};

// A [rows, dim] operand (p may be NULL): resolves its stride and extent.
int check_rows(const void* p, int64_t stride, int64_t es, int64_t rows, int64_t dim, Rows* out) {
  if (stride != 0 && (stride < dim || stride > ((int64_t)1 << 28))) return KDA_ERR_SHAPE;
  if (p && !aligned(p, (uintptr_t)es)) return KDA_ERR_ALIGN;
  out->p = p;
  out->stride = stride == 0 ? dim : stride;
  out->es = es;
  out->set = kda::row_set(p, rows, out->stride, dim, es);
  return KDA_OK;
}

// Whether output `o` may not be where input `i` is: it may be exactly there
// when `exact` (the same rows, element for element), and nowhere else.
bool clash(const Rows& o, const Rows& i, bool exact) {
  if (!overlap(o.set, i.set)) return false;
  return !(exact && o.p == i.p && o.stride == i.stride && o.es == i.es);
}

int check_common(int32_t dtype, int32_t dim, int32_t gate, float eps, int64_t rows) {
  if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (dim < 1 || dim > kMaxDim || rows < 0 || rows > INT32_MAX) return KDA_ERR_SHAPE;
  if (gate != KDA_NORM_GATE_LINEAR && gate != KDA_NORM_GATE_SILU && gate != KDA_NORM_GATE_SIGMOID)
    return KDA_ERR_UNSUPPORTED;
  if (!(std::isfinite(eps) && eps >= 0.f)) return KDA_ERR_SHAPE;
  return KDA_OK;
}

}  // namespace

extern "C" {

int kda_gated_norm(const kda_gated_norm_desc* d, void* stream) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_gated_norm_desc)) return KDA_ERR_VERSION;
  int st = check_common(d->dtype, d->dim, d->gate, d->eps, d->rows);
  if (st != KDA_OK) return st;
  if (d->gate_first != 0 && d->gate_first != 1) return KDA_ERR_UNSUPPORTED;
  const int64_t es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4;
  Rows x, z, y;
  if ((st = check_rows(d->x, d->x_stride, es, d->rows, d->dim, &x)) != KDA_OK ||
      (st = check_rows(d->z, d->z_stride, es, d->rows, d->dim, &z)) != KDA_OK ||
      (st = check_rows(d->y, d->y_stride, es, d->rows, d->dim, &y)) != KDA_OK)
    return st;
  if (!aligned(d->weight, 4)) return KDA_ERR_ALIGN;
  if (d->rows == 0) return KDA_OK;
  if (!d->x || !d->y) return KDA_ERR_NULL;
  if (clash(y, x, true) || clash(y, z, true) ||
      overlap(range_of(y.set), range_of(d->weight, d->weight ? (int64_t)d->dim * 4 : 0)))
    return KDA_ERR_ALIAS;
  kda::GatedNormArgs a;
  a.bf16 = es == 2;
  a.dim = d->dim;
  a.gate = d->gate;
  a.gate_first = d->gate_first == 1;
  a.eps = d->eps;
  a.rows = d->rows;
  a.x = d->x;
  a.w = d->weight;
  a.z = d->z;
  a.y = d->y;
  a.xs = x.stride;
  a.zs = z.stride;
  a.ys = y.stride;
  return kda::hip_status(kda::launch_gated_norm(a, (hipStream_t)stream));
}

int kda_block_norm(const kda_block_norm_desc* d, void* stream) {
  if (!d) return KDA_ERR_NULL;
  if (d->struct_size != sizeof(kda_block_norm_desc)) return KDA_ERR_VERSION;
  int st = check_common(d->dtype, d->dim, d->gate, d->eps, d->rows);
  if (st != KDA_OK) return st;
  const int32_t rd = d->residual_dtype == 0 ? d->dtype : d->residual_dtype;
  if (rd != KDA_DTYPE_F32 && rd != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (rd == KDA_DTYPE_BF16 && d->dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  if (!std::isfinite(d->scale)) return KDA_ERR_SHAPE;
  const int64_t es = d->dtype == KDA_DTYPE_BF16 ? 2 : 4, rs = rd == KDA_DTYPE_BF16 ? 2 : 4;
  Rows x, z, r, ro, y;
  if ((st = check_rows(d->x, d->x_stride, es, d->rows, d->dim, &x)) != KDA_OK ||
      (st = check_rows(d->z, d->z_stride, es, d->rows, d->dim, &z)) != KDA_OK ||
      (st = check_rows(d->r, d->r_stride, rs, d->rows, d->dim, &r)) != KDA_OK ||
      (st = check_rows(d->r_out, d->r_out_stride, rs, d->rows, d->dim, &ro)) != KDA_OK ||
      (st = check_rows(d->y, d->y_stride, es, d->rows, d->dim, &y)) != KDA_OK)
    return st;
  const float* ws[] = {d->w_post, d->w_pre, d->c};
  for (const float* w : ws)
    if (!aligned(w, 4)) return KDA_ERR_ALIGN;
  if (d->rows == 0) return KDA_OK;
  if (!d->x || !d->r || !d->r_out || (d->w_pre != nullptr) != (d->y != nullptr)) return KDA_ERR_NULL;
  if (clash(ro, r, true) || clash(ro, x, false) || clash(ro, z, false) || clash(ro, y, false) ||
      clash(y, x, true) || clash(y, z, true) || clash(y, r, false))
    return KDA_ERR_ALIAS;
  for (const float* w : ws) {
    const Range rw = range_of(w, w ? (int64_t)d->dim * 4 : 0);
    if (overlap(range_of(ro.set), rw) || overlap(range_of(y.set), rw)) return KDA_ERR_ALIAS;
  }
  kda::BlockNormArgs a;
  a.bf16 = es == 2;
  a.res_bf16 = rs == 2;
  a.dim = d->dim;
  a.gate = d->gate;
  a.eps = d->eps;
  a.scale = d->scale;
  a.rows = d->rows;
  a.x = d->x;
  a.r = d->r;
  a.w_post = d->w_post;
  a.w_pre = d->w_pre;
  a.c = d->c;
  a.z = d->z;
  a.r_out = d->r_out;
  a.y = d->y;
  a.xs = x.stride;
  a.rs = r.stride;
  a.zs = z.stride;
  a.ros = ro.stride;
  a.ys = y.stride;
  return kda::hip_status(kda::launch_block_norm(a, (hipStream_t)stream));
}

}  // extern "C"
