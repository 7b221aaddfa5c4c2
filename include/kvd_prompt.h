/*
 * kvd_prompt.h -- the prompt path of libkvd.so: rotary positions, ragged
 * writes into and reads from the paged cache, and attention of several new
 * tokens a sequence over a cache held in 4 bits.
 *
 * A prompt, a chunk of one or a few speculated tokens run through these
 * calls in the order of a layer: kvd_kv_write (which rotates the new
 * queries and keys and encodes keys and values into the cache), then
 * kvd_gqa_extend (whose queries attend to everything up to themselves).
 * Single new tokens are the case of one row a sequence. The conventions of
 * kvd.h hold: device pointers, asynchronous on `stream`, arguments checked
 * on the host before anything is launched, device-resident values checked
 * by the kernels and flagged in the device error word.
 */
#ifndef KVD_PROMPT_H
#define KVD_PROMPT_H

#include "kvd.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Rows of a ragged batch: bf16 vectors (row, head) of one width, element i
 * of them at data[row * row_stride + head * head_stride + i]. The strides
 * are in elements, so the query, key and value parts of a fused projection
 * are passed where they lie. Rows `row_start[b] .. row_start[b + 1] - 1`
 * (device int32 [batch + 1], ascending) belong to sequence b; rows from
 * row_start[batch] on are padding: not read, and left as they were.
 * A sequence that starts below 0 or ends past `rows` is skipped, as if its
 * rows were padding, and KVD_DEVERR_LEN is set. So it is by a list that
 * descends somewhere: kvd_kv_write and kvd_kv_read then do nothing (with more
 * than 2,048 sequences they go on, and which sequence a row is taken for is
 * unspecified); kvd_gqa_extend skips the sequence whose entries descend and
 * all behind it.
 */
typedef struct kvd_rows {
  void *data;
  int32_t rows;
  int32_t heads;
  int64_t row_stride;
  int64_t head_stride;
} kvd_rows;

/*
 * Rotary positions of one to four axes (text: the token's index; images and
 * video: time, height and width). The first d_rot channels of a head are
 * d_rot / 2 pairs; pair i belongs to one axis and turns by
 *     angle_i = positions[axis_i][row] * f_i   radians,
 *     (a, b) -> (a cos - b sin, b cos + a sin),
 * channels from d_rot on stay. Frequencies are passed as fractions of a
 * turn, turns_i = f_i / (2 pi) modulo 1 in units of 2^-64 (kvd_rope_turns):
 * position times turns_i wraps exactly at whole turns, so an angle is as
 * exact at position 2^31 - 1 as at 1.
 *   turns    device uint64 [d_rot / 2]
 *   axis     device uint8 [d_rot / 2]: each pair's axis, or NULL (axis 0).
 *            An entry >= n_axes is taken as axis 0 and flagged
 *            KVD_DEVERR_INDEX
 *   d_rot    even, at most the head width
 *   n_axes   1 .. 4
 *   pairing  KVD_PAIR_HALF: channels i and i + d_rot / 2 make pair i;
 *            KVD_PAIR_ADJACENT: channels 2i and 2i + 1
 *   inverse  0, or 1 to turn by -angle (undoes the rotation; also its
 *            gradient, the transposed rotation)
 */
typedef enum kvd_pairing { KVD_PAIR_HALF = 0, KVD_PAIR_ADJACENT = 1 } kvd_pairing;
typedef struct kvd_rope_plan {
  const uint64_t *turns;
  const uint8_t *axis;
  int32_t d_rot;
  int32_t n_axes;
  int32_t pairing; /* kvd_pairing */
  int32_t inverse;
} kvd_rope_plan;

/*
 * kvd_rope_turns -- HOST: the turns of n frequencies in radians per
 * position (finite, |f| < 2^31; negative ones turn backwards), both HOST
 * arrays. Errors: KVD_ERR_NULL, KVD_ERR_SHAPE.
 */
kvd_status kvd_rope_turns(const double *freq, int32_t n, uint64_t *turns);

/*
 * kvd_rope -- rotate the heads of q and of k ("KV cache", "Two tensors per
 * layer": keys are cached after their positions are applied).
 *   positions    device int32 [n_axes][rows], axis a of row r at
 *                positions[a * axis_stride + r]; any int32
 *   head_dim     width of every row, >= d_rot
 *   q, q_out     rows x heads of one shape; q_out may be q itself (the same
 *                data and strides) and must not overlap it otherwise
 *   k, k_out     the same for the keys, as many rows as q, or both NULL
 * Products and sums in fp32, one rounding to bf16. Errors: KVD_ERR_NULL,
 * KVD_ERR_SHAPE (odd d_rot, shapes that differ, output rows that overlap
 * one another), KVD_ERR_UNSUPPORTED (d_rot above 1024, n_axes above 4).
 */
kvd_status kvd_rope(const kvd_rope_plan *plan, const int32_t *positions,
                    int64_t axis_stride, int32_t head_dim, const kvd_rows *q,
                    const kvd_rows *q_out, const kvd_rows *k,
                    const kvd_rows *k_out, kvd_stream stream);

/*
 * kvd_kv_write -- write a ragged batch of new rows into the cache: a prompt,
 * a chunk of one, or one token a sequence. Row row_start[b] + i goes to
 * position start[b] + i of sequence b, encoded as kvd_kv_append encodes a
 * row. With `rope` the keys are rotated first and rounded to bf16 (the
 * cache holds what kvd_rope followed by this call without `rope` would
 * leave), and so are the queries q into q_out when given (no other call
 * needs to run between a projection and the attention).
 *   start        device int32 [batch]
 *   row_start    device int32 [batch + 1] (see kvd_rows)
 *   k_new, v_new rows x n_kv; v_new NULL for a K-only cache. 16-byte
 *                aligned, strides multiples of 8
 *   rope         NULL, or the plan; positions and axis_stride as kvd_rope
 *   q, q_out     only with rope: as kvd_rope, or both NULL
 * No two rows may name the same slot. Errors: those of kvd_kv_append and of
 * kvd_rope; KVD_ERR_UNSUPPORTED when a head of keys and its angles do not fit
 * in shared memory (with rope: 2 head_dim + 4 d_rot above 204,784 bytes). A
 * position outside the block table or a bad block id skips that row and sets
 * KVD_DEVERR_POS / KVD_DEVERR_BLOCK; for row lists see kvd_rows.
 */
kvd_status kvd_kv_write(const kvd_cache *cache, const int32_t *block_table,
                        int32_t max_blocks_per_seq, const int32_t *start,
                        const int32_t *row_start, int32_t batch,
                        const kvd_rows *k_new, const kvd_rows *v_new,
                        const kvd_rope_plan *rope, const int32_t *positions,
                        int64_t axis_stride, const kvd_rows *q,
                        const kvd_rows *q_out, kvd_stream stream);

/*
 * kvd_kv_read -- the converse: positions start[b] .. of sequence b as bf16
 * rows row_start[b] .. row_start[b + 1] - 1 of k_out and v_out (to move a
 * context, to encode it again, or for attention elsewhere). bf16 and MXFP4
 * values are exact; fp8 rows are code * scale in fp32, rounded once.
 *   k_out, v_out rows x n_kv; either may be NULL. 16-byte aligned, strides
 *                multiples of 8
 * Errors as kvd_kv_write. A row whose position or block id is out of range
 * is flagged and left as it was; for row lists see kvd_rows.
 */
kvd_status kvd_kv_read(const kvd_cache *cache, const int32_t *block_table,
                       int32_t max_blocks_per_seq, const int32_t *start,
                       const int32_t *row_start, int32_t batch,
                       const kvd_rows *k_out, const kvd_rows *v_out,
                       kvd_stream stream);

/*
 * kvd_gqa_extend -- attention of the new tokens of every sequence over an
 * MXFP4 cache that already holds them (kvd_kv_write first): prompts, chunks
 * of prompts, speculated tokens, or one token a sequence. Sequence b has
 * n_b = row_start[b + 1] - row_start[b] query rows and T_b =
 * seqs->seq_lens[b] cached positions; its row i sits at position p = T_b -
 * n_b + i and attends to positions
 *     [max(0, s_b, p + 1 - W), p]
 * (s_b and W: seqs->window_start and seqs->window, W = 0 for no window). A
 * row that sees nothing gives out = 0 and lse = -inf.
 *   row_start device int32 [batch + 1] (see kvd_rows), or NULL: row b is
 *             the one new token of sequence b
 *   max_rows  host: an upper bound on every n_b, 1 without row_start. It
 *             chooses the kernel, for all sequences alike, and sizes the
 *             workspace. Single tokens beside a long chunk are faster in a
 *             call of their own (1,021 rows over 32,000 positions and 32 single
 *             tokens over 8,192, 64 heads: 1,270 us in one call, 1,018 and 76
 *             in two)
 *   q         rows x n_h, head_dim wide, 16-byte aligned, strides multiples
 *             of 8; head h reads KV head h / (n_h / n_kv)
 *   scale     softmax scale; <= 0 selects 1/sqrt(head_dim)
 *   out       device bf16 [rows][n_h][head_dim], 16-byte aligned; must not
 *             overlap q (else KVD_ERR_SHAPE: parts of a row block read q while
 *             others write)
 *   lse       device fp32 [rows][n_h] or NULL
 *   workspace at least kvd_extend_workspace_size() bytes, 256-byte aligned
 *             (NULL when that is 0); see "Workspace" in kvd.h
 * Rows from row_start[batch] on, and those of sequences that are skipped (see
 * kvd_rows), are left as they were. A sequence of more than max_rows rows is
 * skipped as well and flagged KVD_DEVERR_LEN. Scores and sums
 * in fp32; the queries enter the first product as f16 with a power-of-two
 * scale per (row, head), the probabilities enter the second as f16 with the
 * largest at 2^7 or above: each is rounded by 2^-11, and n of them that are
 * 2^-32 of the largest or less lose up to n 2^-32 of the weight. A query
 * that is not finite stays in its own (row, head). The writing calls store
 * finite groups only; where a caller's own bytes hold a NaN scale of V, rows
 * of the same sequence that do not see the position may become NaN as well.
 * Supported: an MXFP4 cache (head_dim 128), n_h / n_kv of 1 .. 128, at most
 * 1024 sequences a call. seqs->flags must be valid and are ignored.
 */
kvd_status kvd_gqa_extend(const kvd_cache *cache, const kvd_seqs *seqs,
                          const int32_t *row_start, int32_t max_rows,
                          const kvd_rows *q, float scale, void *out,
                          float *lse, void *workspace,
                          size_t workspace_bytes, kvd_stream stream);

/* Workspace bytes of a kvd_gqa_extend call with these arguments (`rows` =
 * q->rows) on the current device; 0 when it needs none. */
kvd_status kvd_extend_workspace_size(const kvd_cache *cache,
                                     const kvd_seqs *seqs, int32_t rows,
                                     int32_t max_rows, int32_t n_h,
                                     size_t *bytes);

#ifdef __cplusplus
}
#endif
#endif /* KVD_PROMPT_H */
