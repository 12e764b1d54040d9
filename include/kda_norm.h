/*
 * kda_norm.h -- C ABI of libkda, part 4: the norms of a layer around the KDA
 * or linear attention step.  Both ops are row-wise; RMSNorm(u; w) of a row u
 * of `dim` values is
 *
 *     u_c / sqrt(mean(u^2) + eps) * w_c
 *
 * with the sum of squares, and everything up to the final rounding, in fp32.
 *
 * Conventions are those of kda.h.  Weights are fp32.  Row strides are in
 * elements (0 = dense, else dim .. 2^28); operands may be slices of one wider
 * buffer.  Every pointer needs the alignment of its elements only.  NaN/Inf
 * propagate within their row.
 */
#ifndef KDA_NORM_H
#define KDA_NORM_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* act(z) of a gate: z, z / (1 + e^-z), 1 / (1 + e^-z). */
typedef enum { KDA_NORM_GATE_LINEAR = 0, KDA_NORM_GATE_SILU = 1, KDA_NORM_GATE_SIGMOID = 2 } kda_norm_gate;

/* The output norm of the recurrence, with its gate.  A row is what is
 * normalised together: one token's head ([T, H, dv] is T * H rows of dv) or a
 * whole token.
 *
 *     gate_first = 0:  y = RMSNorm(x; w) * act(z)
 *     gate_first = 1:  y = RMSNorm(x * act(z); w)
 *
 * z = NULL: no gate (the plain RMSNorm).  y may be exactly x or z (in place,
 * with the same stride) and may not partly overlap an input. */
typedef struct {
  uint32_t struct_size;         /* sizeof(kda_gated_norm_desc)                  */
  int32_t dtype;                /* kda_dtype of x, z, y                         */
  int32_t dim;                  /* 1 .. 16384                                   */
  int32_t gate;                 /* kda_norm_gate                                */
  int32_t gate_first;           /* 0 or 1                                       */
  float eps;                    /* >= 0                                         */
  int64_t rows;                 /* 0 .. 2^31 - 1                                */
  const void* x;
  const float* weight;          /* [dim]; NULL = ones                           */
  const void* z;                /* NULL = no gate                               */
  void* y;
  int64_t x_stride, z_stride, y_stride;
} kda_gated_norm_desc;

/* The norms around a block: its output x joins the residual stream r, and the
 * next block's input y is the norm of the sum.
 *
 *     p  = RMSNorm(x; w_post)                 (w_post NULL: p = x)
 *     r' = r + scale * c * act(z) * p         (c NULL: 1; z NULL: no gate)
 *     y  = RMSNorm(r'; w_pre)                 (w_pre NULL: no y)
 *
 * y is computed from r' before r' is rounded to its storage type.  The
 * residual is fp32, or bf16 with bf16 x.  r_out may be exactly r, y exactly x
 * or z (in place, same stride); no output may partly overlap an input or the
 * other output. */
typedef struct {
  uint32_t struct_size;         /* sizeof(kda_block_norm_desc)                  */
  int32_t dtype;                /* kda_dtype of x, z, y                         */
  int32_t residual_dtype;       /* kda_dtype of r, r_out; 0 = dtype             */
  int32_t dim;                  /* 1 .. 16384                                   */
  int32_t gate;                 /* kda_norm_gate                                */
  float eps;                    /* >= 0                                         */
  float scale;
  int64_t rows;                 /* 0 .. 2^31 - 1                                */
  const void* x;
  const void* r;
  const float* w_post;          /* [dim] or NULL                                */
  const float* w_pre;           /* [dim] or NULL                                */
  const float* c;               /* [dim] or NULL                                */
  const void* z;                /* NULL = no gate                               */
  void* r_out;
  void* y;                      /* required exactly when w_pre is given         */
  int64_t x_stride, r_stride, z_stride, r_out_stride, y_stride;
} kda_block_norm_desc;

int kda_gated_norm(const kda_gated_norm_desc* d, void* stream);
int kda_block_norm(const kda_block_norm_desc* d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_NORM_H */
