/*
 * kvd_tree.h -- attention of several rows a sequence that is not causal,
 * over the paged cache of libkvd.so: trees of drafted tokens, and an
 * encoder's states.
 *
 * A step that verifies drafted trees runs through these calls in this
 * order: kvd_tree_plan once (each node's ancestors and its position); per
 * layer kvd_kv_write (kvd_prompt.h: the nodes' keys and values behind the
 * cached context, rotated to the plan's positions) and kvd_gqa_tree; and,
 * when the accepted path of every tree is known, kvd_kv_keep once for all
 * layers. Cross attention is kvd_gqa_cross over a cache that kvd_kv_write
 * filled with the encoder's keys and values once.
 *
 * The conventions of kvd.h hold: device pointers, asynchronous on `stream`,
 * arguments checked on the host before anything is launched, device-resident
 * values checked by the kernels and flagged in the device error word.
 *
 * Row lists (`row_start`, see kvd_rows in kvd_prompt.h) are followed up to
 * their first descent: the sequence whose entries descend and all behind it
 * are skipped, and so is a sequence of more than max_rows rows or one that
 * the rows do not hold. Skipped sequences are flagged KVD_DEVERR_LEN, their
 * rows and rows from row_start[batch] on are left as they were.
 */
#ifndef KVD_TREE_H
#define KVD_TREE_H

#include "kvd_prompt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Nodes of a tree, at most. */
#define KVD_TREE_NODES 256

/*
 * kvd_tree_plan -- trees of drafted tokens from their parents: node i of
 * sequence b is row row_start[b] + i, its parent node parents[row] of the
 * same sequence, with parents[row] < i, or -1 for a node that follows the
 * context itself. Its depth is the number of its ancestors.
 *   start      device int32 [batch]: the cached length before the tree
 *   rows       rows of parents, masks and positions
 *   max_rows   host: an upper bound on every sequence's nodes, at most
 *              KVD_TREE_NODES
 *   window     0, or W > 0: ancestors W or more levels up are left out (for
 *              kvd_gqa_tree with that window)
 *   masks      device uint32 [rows][(max_rows + 31) / 32]: bit j % 32 of word
 *              j / 32 is set for the node itself and its ancestors j
 *   positions  device int32 [rows] or NULL: start[b] + depth, the position
 *              that the node's query and key are rotated to
 * A parent outside [-1, i) is taken as -1 and flagged KVD_DEVERR_INDEX.
 * Errors: KVD_ERR_NULL, KVD_ERR_SHAPE, KVD_ERR_UNSUPPORTED (max_rows above
 * KVD_TREE_NODES, more than 1024 sequences).
 */
kvd_status kvd_tree_plan(const int32_t *parents, const int32_t *start,
                         const int32_t *row_start, int32_t batch, int32_t rows,
                         int32_t max_rows, int32_t window, uint32_t *masks,
                         int32_t *positions, kvd_stream stream);

/*
 * kvd_gqa_tree -- attention of the drafted nodes of every sequence over a
 * cache that holds them (kvd_kv_write first). Sequence b has n_b =
 * row_start[b + 1] - row_start[b] nodes and T_b = seqs->seq_lens[b] cached
 * positions: the context [0, T_b - n_b), and node j at position T_b - n_b +
 * j. Its row i attends to
 *   the context from max(s_b, positions[row] + 1 - W) on, and
 *   the nodes j < n_b whose bit of masks[row] is set
 * (s_b and W: seqs->window_start and seqs->window, W = 0 for no window). The
 * masks may be any, not only those of a tree; a row that sees nothing gives
 * out = 0 and lse = -inf.
 *   row_start  device int32 [batch + 1]
 *   max_rows   host: an upper bound on every n_b, 1 .. KVD_TREE_NODES
 *   q          rows x n_h, head_dim wide, 16-byte aligned, strides multiples
 *              of 8; head h reads KV head h / (n_h / n_kv)
 *   masks      device uint32 [rows][(max_rows + 31) / 32] (kvd_tree_plan)
 *   positions  device int32 [rows], read with a window only (else NULL)
 *   scale      softmax scale; <= 0 selects 1/sqrt(head_dim)
 *   out        device bf16 [rows][n_h][head_dim], 16-byte aligned; must not
 *              overlap q (else KVD_ERR_SHAPE)
 *   lse        device fp32 [rows][n_h] or NULL
 *   workspace  at least kvd_attend_workspace_size() bytes, 256-byte aligned
 *              (NULL when that is 0); see "Workspace" in kvd.h
 * A sequence with T_b < n_b is skipped and flagged KVD_DEVERR_LEN. positions
 * below T_b - n_b are taken as that. Scores and sums in fp32; the probabilities
 * enter the second product as bf16 (bf16 caches) or f16, each rounded by half a
 * step. Positions that no row of a sequence sees (nodes that no mask has,
 * context before every row's window) may hold anything; a value of V that is
 * not finite, at a position that some row of the sequence sees, may show in
 * rows that see other positions only (rows that see nothing stay 0).
 * Supported: bf16 and fp8 caches with head_dim 64 or 128 and MXFP4 caches,
 * n_h / n_kv of 1 .. 128, at most 1024 sequences a call, bf16 caches of less
 * than 2^31 rows (blocks x heads x slots), lengths up to 2^31 - 256. K and V of a
 * bf16 cache that lie 2^40 bytes or more apart must both be device memory (else
 * KVD_ERR_UNSUPPORTED). seqs->flags must be valid and are ignored.
 */
kvd_status kvd_gqa_tree(const kvd_cache *cache, const kvd_seqs *seqs,
                        const int32_t *row_start, int32_t max_rows,
                        const kvd_rows *q, const uint32_t *masks,
                        const int32_t *positions, float scale, void *out,
                        float *lse, void *workspace, size_t workspace_bytes,
                        kvd_stream stream);

/*
 * kvd_gqa_cross -- attention of rows to another sequence's states, held in
 * the cache: every row of sequence b attends to the positions [max(0, s_b),
 * seqs->seq_lens[b]) alike (s_b: seqs->window_start, 0 without; inputs padded
 * on the left start there). seqs->window must be 0. A row that sees nothing
 * gives out = 0 and lse = -inf.
 *   row_start  device int32 [batch + 1], or NULL: row b is the one row of
 *              sequence b (max_rows 1)
 *   max_rows   host: an upper bound on the rows of a sequence; it sizes the
 *              workspace
 *   other arguments and supported shapes as kvd_gqa_tree
 * Without row_start this is what kvd_gqa_decode computes with window_start =
 * s_b, for every group size and width here. For the shapes that both take,
 * kvd_gqa_decode is faster where there are many kv heads and this call where
 * there are few with groups of 2 and more (16 sequences of 1,060 states, us, this
 * / that: 16 heads of 16 kv heads, head_dim 64, bf16 31 / 20, fp8 40 / 19; 32 of
 * 32, 128, bf16 65 / 49; 32 of 8, 128, bf16 22 / 30, MXFP4 20 / 30; 64 of 8, 128,
 * bf16 22 / 23); for groups of 1, 2 and 4 kvd_gqa_decode keeps the
 * probabilities in fp32.
 */
kvd_status kvd_gqa_cross(const kvd_cache *cache, const kvd_seqs *seqs,
                         const int32_t *row_start, int32_t max_rows,
                         const kvd_rows *q, float scale, void *out, float *lse,
                         void *workspace, size_t workspace_bytes,
                         kvd_stream stream);

/* Workspace bytes of a kvd_gqa_tree or kvd_gqa_cross call with these arguments
 * (`rows` = q->rows, `lists`: 0 for a kvd_gqa_cross without row_start) on the
 * current device; 0 when it needs none. */
kvd_status kvd_attend_workspace_size(const kvd_cache *cache,
                                     const kvd_seqs *seqs, int32_t rows,
                                     int32_t max_rows, int32_t n_h,
                                     int32_t lists, size_t *bytes);

/*
 * kvd_kv_keep -- after a tree's verification: the cached rows of its accepted
 * nodes move behind the context. In every cache of the list, position
 * start[b] + j of sequence b takes the row of position start[b] + path[b][j],
 * for j < n_keep[b]; nothing else changes (the caller's new length is
 * start[b] + n_keep[b]).
 *   caches     HOST array of n_caches caches (the layers') of one shape and
 *              type, K and V or all K-only; neither a cache nor a tensor of
 *              one may be listed twice (but K and V may be one tensor)
 *   start      device int32 [batch]
 *   path       device int32 [batch][width], a sequence's accepted nodes from
 *              the root on: ascending (a node follows its parent), from 0 up
 *   n_keep     device int32 [batch]: 0 .. width
 * A sequence whose path is not strictly ascending from 0 or more is left as
 * it was and flagged KVD_DEVERR_INDEX, one whose n_keep is outside [0, width]
 * KVD_DEVERR_LEN, one with a position outside the block table KVD_DEVERR_POS
 * or a bad block id KVD_DEVERR_BLOCK. No block that receives a row may be
 * shared with another sequence of the call. Errors: KVD_ERR_NULL,
 * KVD_ERR_SHAPE (caches that differ), KVD_ERR_UNSUPPORTED (width above
 * KVD_TREE_NODES, more than 1024 sequences).
 */
kvd_status kvd_kv_keep(const kvd_cache *caches, int32_t n_caches,
                       const int32_t *block_table, int32_t max_blocks_per_seq,
                       const int32_t *start, const int32_t *path,
                       int32_t width, const int32_t *n_keep, int32_t batch,
                       kvd_stream stream);

#ifdef __cplusplus
}
#endif
#endif /* KVD_TREE_H */
