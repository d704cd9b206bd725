/*
 * bfp8_attention.h -- C ABI of libbfp8, second part: what a decoder layer
 * computes between its QKV projection and its output projection, forward and
 * backward.  The conventions of bfp8.h hold: plain device pointers and sizes,
 * every argument validated on the host before any HIP call, a bfp8_status
 * returned, all work enqueued on the given stream, nothing allocated, no
 * state kept, no synchronisation.  Results are deterministic: no atomics, and
 * every sum has one fixed order.
 *
 * The Puro-2B recipe keeps the attention core in BF16 beside the FP8 linear
 * layers (Puro-2B tutorial, FP8/MuonH section; Puro-2B paper, zh-TW
 * translation, section 2), with 16 query and 8 key/value heads of 128.
 *
 * Tensors of heads.  A tensor [tokens][heads][head_dim] is given by its first
 * element and two strides in elements: `row` from token to token and `head`
 * from head to head; the head_dim values of one head are contiguous.  So the
 * q, k and v heads of a fused projection's rows, tensors stored head by head
 * and caches are all taken as they lie.  Pointers are 16-byte aligned, strides
 * keep every head 16-byte aligned, and row strides are at most 2^22 elements.
 *
 * Sizes.  A call whose launch would need 2^32 threads or more is refused with
 * BFP8_ERR_SHAPE: a rotation of 2^29 heads in all (of 128 bf16 values in 16-byte
 * units, 2^24 at the least), a table of 2^32 pairs, attention of about 2^31 rows
 * (tokens times query heads), its gradient of 2^28 rows or 2^30 keys (tokens
 * times kv heads).
 */
#ifndef BFP8_ATTENTION_H_
#define BFP8_ATTENTION_H_

#include "bfp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions ------------------------------------------------------
 *
 * Pair i of a head's first rot_dim values turns by the angle p * f_i of its
 * token's position p:
 *   y_a = c x_a - s x_b,  y_b = s x_a + c x_b,
 *   c = m cos(p f_i),  s = m sin(p f_i),  i = 0 .. rot_dim/2 - 1.
 * BFP8_ROPE_HALF pairs (i, i + rot_dim/2); BFP8_ROPE_INTERLEAVED (2i, 2i+1).
 * Values past rot_dim are copied.
 *
 * Frequencies f_i = base^(-2i/rot_dim), m = 1, changed for long contexts by
 *   BFP8_ROPE_LINEAR  f_i / factor  (positions interpolated);
 *   BFP8_ROPE_NTK     base * factor^(rot_dim/(rot_dim-2)) in place of base
 *                     (rot_dim 2, whose one frequency is 1, stays as it is);
 *   BFP8_ROPE_YARN    g_i f_i + (1 - g_i) f_i / factor,
 *                     g_i = clamp((t_i - 1) / 31, 0, 1) with t_i =
 *                     original_length * f_i / (2 pi) the turns a pair makes
 *                     over the original context; m = 0.1 ln(factor) + 1.  (The
 *                     ramp is linear in the turns, from 1 to 32; models whose
 *                     program ramps over the pair's index, or between other
 *                     bounds, need another table of the same layout.)
 */
typedef enum { BFP8_ROPE_HALF = 0, BFP8_ROPE_INTERLEAVED = 1 } bfp8_rope_layout;
typedef enum {
  BFP8_ROPE_NONE = 0,
  BFP8_ROPE_LINEAR = 1,
  BFP8_ROPE_NTK = 2,
  BFP8_ROPE_YARN = 3
} bfp8_rope_scaling;

/* table [positions][rot_dim/2][2] float32: (m cos, m sin) of positions 0 ..
 * positions-1, angles taken in float64.  rot_dim even and > 0, base > 0,
 * factor >= 1 (unused with BFP8_ROPE_NONE), original_length > 0 with
 * BFP8_ROPE_YARN (unused otherwise); BFP8_ERR_SHAPE if not, BFP8_ERR_LAYOUT
 * for an unknown scaling. */
bfp8_status bfp8_rope_table(float* table, int64_t positions, int rot_dim, double base,
                            bfp8_rope_scaling scaling, double factor, int64_t original_length,
                            hipStream_t stream);

/* y = x turned, for x, y [tokens][heads][head_dim] of dtype dt.  y may be x
 * itself (same pointer and strides); any other overlap is not allowed.
 *   table      [table_rows][rot_dim/2][2] from bfp8_rope_table
 *   positions  int32 [tokens], or NULL: token t stands at position t.  A
 *              token whose position is outside [0, table_rows) gets NaN in
 *              its turned values, but a pair of zeros stays zero: so padding
 *              may stand at any position, -1 among them.
 *   inverse    0, or 1: turns by -p f_i, which is the gradient: dx from dy
 *              (the transpose of the turn, so the factor m stays).
 * head_dim * (size of dt) is a multiple of 16 bytes; rot_dim is even and
 * 0 < rot_dim <= head_dim.  BFP8_ERR_LAYOUT for an unknown layout. */
bfp8_status bfp8_rope(const void* x, int64_t x_row, int64_t x_head, void* y, int64_t y_row,
                      int64_t y_head, bfp8_in_dtype dt, int64_t tokens, int64_t heads,
                      int head_dim, int rot_dim, bfp8_rope_layout layout, const float* table,
                      int64_t table_rows, const int32_t* positions, int inverse,
                      hipStream_t stream);

/* ---- attention -------------------------------------------------------------
 *
 * For each sequence b and query head h, with g = h / (heads / kv_heads):
 *   S = scale Q_h K_g^T,  O_h = softmax(S) V_g,  L_h = ln sum_j exp S_j.
 * With `causal`, query i of n sees keys 0 .. i + m - n of m (the last query
 * sees every key).  A query that sees no key gets O = 0 and L = -inf, and
 * gradients of zero.  All tensors bf16 and 16-byte aligned per head, L
 * float32 [heads][total_q]; products of bf16 values are summed in float32,
 * the softmax's maximum and sum are float32, and the probabilities (and, for
 * the gradients, dS) are rounded to bf16 for their products only.  Values of
 * other sequences, and of rows past a sequence's used length, are never part
 * of a result, whatever they hold; Inf or NaN within a sequence's own used
 * rows is outside the contract (no fault, but any row of that sequence may be
 * affected; a query with a NaN score gets NaN in O and L).  With BFP8_DEBUG (see
 * bfp8.h) q, dout and, without k_lens, k and v are scanned whole, rows of no
 * sequence among them.
 *
 * Sequences lie one after another in the tensors' rows:
 *   cu_q [batch+1], cu_k [batch+1]  int32 device arrays, non-decreasing:
 *       sequence b has rows cu[b] .. cu[b+1]-1.  NULL: batch sequences of
 *       total/batch rows each (total divisible by batch).
 *   k_lens [batch]  int32 device array or NULL: only the first k_lens[b] key
 *       rows of sequence b are used (a cache with room).
 * The host cannot see these arrays: the kernels clamp every entry into the
 * tensors' rows, so no entry makes them read or write elsewhere.
 *
 * Rows before cu[0] and from cu[batch] on belong to no sequence.  A result
 * keeps what it held there, unless the bit added to `causal` names it: then it is
 * 0 (L: -inf).
 */
enum {
  BFP8_CLEAR_O = 1 << 8, /* of the forward call */
  BFP8_CLEAR_LSE = 1 << 9,
  BFP8_CLEAR_DQ = 1 << 10, /* of the backward call */
  BFP8_CLEAR_DK = 1 << 11,
  BFP8_CLEAR_DV = 1 << 12
};
typedef struct {
  int64_t batch;
  int64_t total_q, total_k; /* rows of q, o, dq, do / of k, v, dk, dv; at most
                               2^31 - 512 together */
  const int32_t* cu_q;
  const int32_t* cu_k;
  const int32_t* k_lens;
  int heads, kv_heads; /* heads a multiple of kv_heads */
  int head_dim;        /* a multiple of 8, at most 128 */
  int causal;          /* 0 or 1, plus BFP8_CLEAR_* of the results to clear */
  float scale;
} bfp8_attention_shape;

/* A tensor of heads: pointer and strides in elements (see the top). */
typedef struct {
  const void* data;
  int64_t row, head;
} bfp8_heads;
typedef struct {
  void* data;
  int64_t row, head;
} bfp8_heads_out;

/* Device memory the calls below use (0: none): backward 0 or 1.  (size_t)-1
 * for an invalid shape. */
size_t bfp8_attention_workspace_bytes(const bfp8_attention_shape* shape, int backward);

/* o and lse, which must not overlap the inputs, from q, k, v.  The workspace
 * holds float32 partial results where the keys of few query rows are split over
 * workgroups; smaller or NULL: no split (same contract, slower). */
bfp8_status bfp8_attention_forward(const bfp8_attention_shape* shape, bfp8_heads q, bfp8_heads k,
                                   bfp8_heads v, bfp8_heads_out o, float* lse, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* dq, dk, dv from the forward pass's inputs, its o and lse, and the gradient
 * dout of o; the probabilities are recomputed from lse.  Rows of dk and dv
 * past a sequence's used length become zero.  The workspace
 * (bfp8_attention_workspace_bytes(shape, 1): two float32 values a row and head,
 * and partial gradients where few workgroups meet long sequences) is required:
 * BFP8_ERR_WORKSPACE if it is NULL or smaller.  dq, dk and dv must not overlap
 * each other or the inputs. */
bfp8_status bfp8_attention_backward(const bfp8_attention_shape* shape, bfp8_heads q, bfp8_heads k,
                                    bfp8_heads v, bfp8_heads o, const float* lse, bfp8_heads dout,
                                    bfp8_heads_out dq, bfp8_heads_out dk, bfp8_heads_out dv,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BFP8_ATTENTION_H_ */
