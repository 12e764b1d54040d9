/*
 * kda_latent.h -- C ABI of libkda, part 5: latent attention and its paged
 * cache, the full-attention layers that stand between the recurrent ones.
 *
 * A latent-attention layer keeps ONE row per token for all its heads: a latent
 * vector c of dc values, and a positional part of dr values (rotated by the
 * token's position, or not at all).  Per head a query meets it in two forms
 * that are equal up to rounding:
 *
 *   expanded  the keys k = W_k c (dn values) and values v = W_v c (dv values)
 *             of each head are formed by a projection; scores
 *             q[:dn] . k + q[dn:] . k_pe, where k_pe is shared by the heads
 *   absorbed  W_k is multiplied into the query (dc values) instead and W_v
 *             into the output; scores q[:dc] . c + q[dc:] . k_pe on the cached
 *             rows, and the weighted mean of the c themselves as output
 *
 * kda_latent_prefill is the expanded form over packed prompts,
 * kda_latent_attend the absorbed one over the pages, for one new token per
 * sequence or for several; kda_latent_append writes new rows into the pages;
 * kda_rotary turns the queries' positional part.
 *
 * Conventions are those of kda.h (struct_size first, device pointers owned by
 * the caller, every check on the host before anything is enqueued, no
 * allocation, no synchronisation, calls re-entrant).  Strides are in elements,
 * multiples of 16 bytes and at most 2^28 (between pages 2^40); 0 = dense.  Alignment: 16 bytes for
 * tensors of dtype, 8 for frequencies, 4 for weights and index tables.  An
 * output overlaps no input, unless a descriptor says otherwise.
 *
 * The cache: a pool of n_pages pages of page_size rows of dc + dr values.
 * Position p of sequence n is row p % page_size of page
 * block_table[n, p / page_size].  seq_lens[n] counts the sequence's rows with
 * its new tokens among them, which are its last ones.  These three tables are
 * read on the device: a position that is negative, past the table's end or on
 * a page outside 0 .. n_pages - 1 has no row; it is not written, and not seen by
 * any query.
 *
 * Numerics: scores, softmax maxima and sums and all products' sums are fp32.
 * With bf16 inputs the softmax weights are rounded to bf16 (relative 2^-8 at
 * most, after their sum is taken) before they multiply the values, which the
 * matrix cores take in one type; with fp32 inputs everything is fp32.  A query that sees no key has output 0.  NaN and
 * infinities in rows that a query does not see do not reach its output; in rows
 * that it sees they do, an infinite value possibly as NaN.
 */
#ifndef KDA_LATENT_H
#define KDA_LATENT_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Expanded attention over packed sequences, causal: query i of a sequence's Lq
 * sees its keys 0 .. Lk - Lq + i (its last query stands beside its last key).
 *
 * Layouts: q [q_total, H, dn + dr]; k [k_total, H, dn]; k_pe [k_total, dr];
 * v [k_total, H, dv]; o [q_total, H, dv].  k and v may be slices of one buffer
 * [k_total, H, dn + dv]: besides the token stride they have a head stride.
 * The token strides of k, k_pe, v and o are at most 2^22, dense or not.
 * cu_seqlens [N + 1] gives the sequences' queries, cu_seqlens_k [N + 1] their
 * keys; NULL: the same as the queries' (k_total == q_total then).  Both are read
 * on the device, clamped to [0, q_total] and [0, k_total]: contents that break
 * the rules (not ascending from 0) give unspecified results but no access out
 * of bounds.  Rows of o outside every sequence are not written. */
typedef struct {
  uint32_t struct_size;        /* sizeof(kda_latent_prefill_desc)               */
  int32_t dtype;               /* kda_dtype of q, k, k_pe, v, o                 */
  int32_t n_seqs;              /* N >= 1 (a batch of none is no call)           */
  int32_t n_heads;             /* H, 1 .. 65535                                 */
  int32_t dn, dr, dv;          /* dn and dv 64 or 128, dr 32 or 64              */
  float scale;                 /* 2^-126 .. 2^127; 0 = (dn + dr)^-1/2           */
  int64_t q_total, k_total;    /* 0 .. 2^31 - 65; (q_total / 128 + N) H < 2^23  */
  const void* q;
  const void* k;
  const void* k_pe;
  const void* v;
  void* o;
  int64_t q_stride, k_stride, k_head_stride, k_pe_stride, v_stride, v_head_stride, o_stride;
  const int32_t* cu_seqlens;   /* device; NULL allowed if N == 1                */
  const int32_t* cu_seqlens_k; /* device or NULL                                */
} kda_latent_prefill_desc;

/* Bytes of device workspace kda_latent_prefill needs: 0 but where the blocks of
 * queries are too few for the GPU and their keys are shared out (depends on sizes
 * only: dtype, n_seqs, n_heads, dn, dr, dv, q_total and k_total; not monotonic in
 * them, so a buffer for several calls has the largest of their sizes).  *status (host, may
 * be NULL) receives the kda_status of the check; 0 is returned when it fails. */
size_t kda_latent_prefill_workspace_bytes(const kda_latent_prefill_desc* d, int* status);

/* workspace: as in kda_latent_attend. */
int kda_latent_prefill(const kda_latent_prefill_desc* d, void* workspace, size_t workspace_bytes,
                       void* stream);

/* Absorbed attention of new tokens over the paged cache, which holds their own
 * rows already: new token i of a sequence's Lq sees positions
 * 0 .. seq_lens[n] - Lq + i.
 *
 * Layouts: q [t_total, H, dc + dr]; o [t_total, H, dc]; cache [n_pages,
 * page_size, dc + dr]; block_table [N, max_pages]; seq_lens [N].  cu_seqlens
 * [N + 1] gives the sequences' new tokens (clamped as above); NULL: one token
 * for each (t_total == N).  Rows of o outside every sequence are not written.  The
 * token stride of o is at most 2^22, dense or not.
 *
 * A query's result depends, bit for bit, on the whole call: the rows are shared
 * out evenly over the GPU, and where a sequence's rows are cut depends on the
 * others' lengths.  How many queries share a workgroup (32 or 64) is chosen by
 * sizes alone, with max_pages * page_size for the sequences' lengths: a
 * table much wider than they are can cost time (a quarter, for four sequences of
 * 8,000 rows and 128 heads), never a result. */
typedef struct {
  uint32_t struct_size;        /* sizeof(kda_latent_attend_desc)                */
  int32_t dtype;               /* kda_dtype of q, cache, o                      */
  int32_t n_seqs;              /* N, 0 (nothing to do) .. 2^24                  */
  int32_t n_heads;             /* H, 1 .. 65535                                 */
  int32_t dc, dr;              /* dc 256 or 512, dr 32 or 64                    */
  int32_t page_size;           /* >= 1; max_pages * page_size <= 2^31 - 257     */
  int32_t max_pages;           /* >= 1: columns of block_table                  */
  int32_t n_pages;             /* >= 0                                          */
  float scale;                 /* 2^-126 .. 2^127                               */
  int64_t t_total;             /* new tokens; t_total H <= 2^31 - 65            */
  const void* q;
  const void* cache;
  void* o;
  int64_t q_stride, page_stride, row_stride, o_stride;
  const int32_t* block_table;  /* device [N, max_pages]                         */
  const int32_t* seq_lens;     /* device [N]                                    */
  const int32_t* cu_seqlens;   /* device [N + 1] or NULL                        */
} kda_latent_attend_desc;

/* Bytes of device workspace kda_latent_attend needs (depends on sizes only:
 * dtype, n_seqs, n_heads, dc, dr, max_pages, page_size, t_total and whether
 * cu_seqlens is NULL; not monotonic in them, so a buffer for several calls has the
 * largest of their sizes).  *status (host, may be NULL) receives the kda_status of
 * the check; 0 is returned when it fails. */
size_t kda_latent_workspace_bytes(const kda_latent_attend_desc* d, int* status);

/* workspace: at least that many bytes (NULL allowed when 0), 256-byte aligned,
 * owned by the caller; calls that may overlap, and graphs that may run at the
 * same time, need one each.  Its contents need not be kept or cleared. */
int kda_latent_attend(const kda_latent_attend_desc* d, void* workspace, size_t workspace_bytes,
                      void* stream);

/* How a positional part is turned by the angle t = position * frequency, with
 * m = magnitude: (a, b) -> m (a cos t - b sin t, b cos t + a sin t). */
typedef enum {
  KDA_ROTARY_HALF = 0,        /* pairs (x[i], x[i + dim / 2])                   */
  KDA_ROTARY_INTERLEAVED = 1  /* pairs (x[2 i], x[2 i + 1])                     */
} kda_rotary_layout;

/* Writes new tokens' rows into the cache: row [RMSNorm(latent) w | R(k_pe)] of
 * new token i of a sequence's Lq at position seq_lens[n] - Lq + i, the rotation
 * by that position.
 *
 * Layouts: latent [t_total, dc], k_pe [t_total, dr] (both may be slices of
 * wider rows), tables as in kda_latent_attend_desc; rows_out [t_total, dc + dr]
 * also receives each token's row where it is not NULL, also of tokens whose
 * position has no row in the cache.  Tokens outside every sequence are not
 * touched.  rows_out may be the buffer that latent and k_pe are slices of, at
 * the same places and strides (one token: at any strides).  Two tokens of one position (a page twice in the
 * table) leave a mixture of their rows. */
typedef struct {
  uint32_t struct_size;        /* sizeof(kda_latent_append_desc)                */
  int32_t dtype;               /* kda_dtype of latent, k_pe, cache, rows_out    */
  int32_t n_seqs;              /* N, 0 (nothing to do) .. 2^24                  */
  int32_t dc, dr;              /* dc 256 or 512, dr 32 or 64                    */
  int32_t page_size, max_pages, n_pages; /* as in kda_latent_attend_desc        */
  int32_t rotary;              /* kda_rotary_layout                             */
  float eps;                   /* >= 0, of the norm                             */
  float magnitude;             /* 0 = 1                                         */
  int64_t t_total;             /* 0 .. 2^25 - 1                                 */
  const void* latent;
  const void* k_pe;
  void* cache;
  void* rows_out;              /* NULL = not returned                           */
  int64_t latent_stride, k_pe_stride, page_stride, row_stride, rows_out_stride;
  const float* weight;         /* [dc], or NULL: latent is written as it is     */
  const double* frequencies;   /* [dr / 2] radians per position, or NULL: k_pe  */
                               /* is written as it is                           */
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_seqlens;   /* device [N + 1]; NULL: one token per sequence  */
} kda_latent_append_desc;

int kda_latent_append(const kda_latent_append_desc* d, void* stream);

/* y = the rows of x turned by their token's position.  x, y [t_total, H, dim]
 * with token and head strides (a slice of wider heads); y may be x itself, or other
 * columns of the same heads.  The
 * angle is formed in fp64 and reduced to one turn before its sine and cosine
 * are taken in fp32 (off by at most 4 half steps of 1), so far positions cost no
 * accuracy. */
typedef struct {
  uint32_t struct_size;        /* sizeof(kda_rotary_desc)                       */
  int32_t dtype;               /* kda_dtype of x, y                             */
  int32_t n_heads;             /* H, 1 .. 65535                                 */
  int32_t dim;                 /* a multiple of 16, 16 .. 256;                  */
                               /* t_total min(H, 8) dim / 4 < 2^31              */
  int32_t rotary;              /* kda_rotary_layout                             */
  float magnitude;             /* 0 = 1                                         */
  int64_t t_total;             /* 0 .. 2^31 - 65                                */
  const void* x;
  void* y;
  int64_t x_stride, x_head_stride, y_stride, y_head_stride;
  const int32_t* positions;    /* device [t_total]                              */
  const double* frequencies;   /* device [dim / 2] radians per position         */
} kda_rotary_desc;

int kda_rotary(const kda_rotary_desc* d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LATENT_H */
