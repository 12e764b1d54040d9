/*
 * kda_linear.h -- C ABI of libkda, part 3: linear attention with one decay
 * per head, the recurrence without the delta rule.
 *
 * Per (sequence, head) a state S with dk rows (key channels) and dv columns
 * (value channels) is carried from token to token.  One token with query q,
 * key k, value v and natural-log decay g (ONE value per head, where KDA has one
 * per key channel) does
 *
 *     S <- exp(g) S + k v^T
 *     o  = scale * S^T q                 (the state after the update)
 *
 * It comes in the two forms KDA has (kda.h): a prefill over packed sequences
 * that returns the final states, and a decode step of one token per sequence
 * on the carried states.
 *
 * Conventions are those of kda.h: struct_size first, device pointers owned by
 * the caller, every check on the host before anything is enqueued, kda_status
 * returns, no allocation, no synchronisation, calls re-entrant, dense
 * row-major tensors whose last index is contiguous.  What differs:
 *   - dk and dv are chosen separately, each in {32, 64, 128}.
 *   - q, k, v and o may have a token stride of their own (a slice of a wider
 *     buffer): the number of elements from one token's first to the next
 *     one's, at least heads * head dim, a multiple of 16 bytes; 0 = dense.
 *     Dense or not, it is at most 2^22.
 *   - Alignment: 16 bytes for q, k, v, o, h0, ht and the decode state; g and
 *     the index tables, 4 bytes.
 *
 * Numerics: states, decays and sums are fp32 or wider (the decays' sums inside
 * a chunk are fp64).  With bf16 inputs the matrix products take bf16 operands:
 * the decayed scores of a chunk and the copy of the state that q is multiplied
 * with are rounded to bf16 (relative 2^-8 at most) on the way to o, while the
 * carried state is updated from products that keep fp32 precision.
 * A log-decay below -200 acts as -200 (exp(-200) is 0 in fp32), so -inf is
 * allowed and forgets the state; NaN propagates.  g > 0 is allowed, but the
 * prefill forms the growth over whole chunks and segments: where that leaves
 * fp32 (past e^88) its results are not finite, also where the state that it
 * multiplies is zero.  A value of q, k, v or g that is not finite reaches the
 * outputs of its own and later tokens of its sequence and head, never earlier
 * ones or another sequence's; an infinite value may arrive there, and in the
 * state, as NaN.
 *
 * A sequence's results depend, bit for bit, on its own data and on the sizes,
 * types and options of the call, which choose the lengths of chunks and
 * segments: not on the sequences packed beside it or on its place among them.
 * In a call of another t_total or N it may be rounded differently.
 */
#ifndef KDA_LINEAR_H
#define KDA_LINEAR_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Decay input: one value per token and head, g [T, H] (decode: [N, H]), or one
 * constant per head, g [H]. */
typedef enum { KDA_DECAY_TOKEN = 0, KDA_DECAY_HEAD = 1 } kda_decay;

/* Prefill over a packed batch of N sequences (t_total tokens).
 *
 * Layouts: q, k [t_total, Hk, dk]; v, o [t_total, H, dv]; g as kda_decay says;
 * h0, ht [N, H, dk, dv] in state_dtype.  Value head h reads key head
 * h / (H / Hk).  An empty sequence writes no o and sets ht = h0 (zeros when h0
 * is NULL).  cu_seqlens as in kda.h; it is read on the device, clamped to
 * [0, t_total]: contents that break the rules give unspecified o and ht but no
 * access out of bounds.  Rows of o outside every sequence are not written.
 *
 * Aliasing: ht may equal h0 (in-place carry), also with state_indices.  o and
 * ht must not overlap any other input or each other. */
typedef struct {
  uint32_t struct_size;         /* sizeof(kda_linear_prefill_desc)              */
  int32_t dtype;                /* kda_dtype of q, k, v, o                      */
  int32_t n_seqs;               /* N >= 1; a call's N * H (and its segments)    */
                                /* stay below 2^24                              */
  int32_t n_heads;              /* H, 1 .. 65535                                */
  int32_t n_k_heads;            /* Hk, dividing H; 0 = H                        */
  int32_t dk, dv;               /* each in {32, 64, 128}                        */
  int32_t decay;                /* kda_decay                                    */
  int64_t t_total;              /* packed tokens, 0 .. 2^31 - 65; v holds fewer */
                                /* than 2^47 values                             */
  float scale;                  /* 0 = dk^-1/2                                  */
  int32_t state_dtype;          /* kda_dtype of h0 and ht; 0 = fp32; bf16 with  */
                                /* bf16 inputs only                             */
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  void* o;
  int64_t q_stride, k_stride, v_stride, o_stride; /* elements per token; 0 = dense */
  const void* h0;               /* NULL = zero initial state                    */
  void* ht;                     /* NULL = final state not returned              */
  const int32_t* cu_seqlens;    /* device int32 [N + 1]; NULL allowed if N == 1 */
  const int32_t* state_indices; /* NULL, or device [N]: h0 and ht are pools     */
                                /* [n_slots, H, dk, dv], sequence n uses slot   */
                                /* state_indices[n]; negative (or >= n_slots)   */
                                /* skips it: no o, no state.  Distinct.         */
  int32_t n_slots;              /* pool size when state_indices is set; n_slots */
                                /* times H at most 2^40                         */
} kda_linear_prefill_desc;

/* One decode step for N sequences.  state [N, H, dk, dv] (or a pool with
 * state_indices) is read and updated IN PLACE; q, k [N, Hk, dk]; v, o
 * [N, H, dv]; g [N, H] or [H].  o must not overlap the state or any input, the
 * state no other input. */
typedef struct {
  uint32_t struct_size;         /* sizeof(kda_linear_decode_desc)               */
  int32_t dtype;                /* kda_dtype of q, k, v, o                      */
  int32_t n_seqs;               /* N >= 0 (0 = nothing to do); N * H < 2^24     */
  int32_t n_heads;              /* H, 1 .. 65535                                */
  int32_t n_k_heads;            /* Hk, dividing H; 0 = H                        */
  int32_t dk, dv;               /* each in {32, 64, 128}                        */
  int32_t decay;                /* kda_decay                                    */
  float scale;                  /* 0 = dk^-1/2                                  */
  int32_t state_dtype;          /* kda_dtype of the state; 0 = fp32             */
  void* state;
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  void* o;
  int64_t q_stride, k_stride, v_stride, o_stride; /* elements per sequence; 0 = dense */
  const int32_t* state_indices; /* as in kda_linear_prefill_desc                */
  int32_t n_slots;
} kda_linear_decode_desc;

/* Bytes of device workspace kda_linear_prefill needs for this descriptor
 * (depends on its sizes only; 0 where it needs none).  *status (host, may be
 * NULL) receives the kda_status of the check; 0 is returned when it fails.
 * A shorter batch may need more than a longer one (its segments are shorter):
 * a buffer for several shapes takes the largest of their sizes. */
size_t kda_linear_workspace_bytes(const kda_linear_prefill_desc* d, int* status);

/* Enqueue the prefill on `stream`.  workspace: device buffer of at least
 * kda_linear_workspace_bytes(d) bytes (NULL allowed when that is 0), 256-byte
 * aligned, owned by the caller; calls that may overlap, and graphs that may
 * run at the same time, need one each. */
int kda_linear_prefill(const kda_linear_prefill_desc* d, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Enqueue one decode step on `stream`. */
int kda_linear_decode(const kda_linear_decode_desc* d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_LINEAR_H */
