// Interface between the C ABI layer (api.cu) and the kernels of the prompt
// path (kvd_prompt.h): parameter structs and launcher functions.
#pragma once

#include "kvd_internal.h"

namespace kvd {

// Rotary positions of a rows_kernel launch (kvd_rope_plan).
struct RopeParams {
  const uint64_t *turns;  // [half]
  const uint8_t *axis;    // [half] or null
  const int32_t *pos;     // [n_axes][rows], axes axis_stride apart
  long axis_stride;
  int32_t half;  // pairs, d_rot / 2
  int32_t n_axes, adjacent, inverse, on;
};

// Ragged rows rotated, written into the cache or read from it (rows.cu).
// Strides in elements: *_rs between rows, *_hs between heads.
constexpr int kMaxRowTile = 16;             // rows a CTA takes at most
constexpr int kRowsMaxSmem = 200 * 1024;
struct RowsParams {
  const uint16_t *q;
  uint16_t *q_out;
  long q_rs, q_hs, qo_rs, qo_hs;
  const uint16_t *k, *v;  // new rows (v null for a K-only cache)
  long k_rs, k_hs, v_rs, v_hs;
  uint16_t *k_out, *v_out;  // rotated keys, or rows read back
  long ko_rs, ko_hs, vo_rs, vo_hs;
  RopeParams rope;
  uint8_t *k_cache, *v_cache;
  const float *k_inv, *v_inv, *k_scale, *v_scale;
  const int32_t *block_table, *start, *row_start;
  int32_t rows, n_h, n_kv, d, dtype;
  int32_t batch, max_blocks, block_size, num_blocks;
  int32_t tile;  // rows per CTA (set by the launcher)
  int *err;
};

// kvd_gqa_extend: several new rows a sequence over an MXFP4 cache. The
// DecodeParams fields it uses keep their meaning (out [rows][n_h][dv], lse
// [rows][n_h]).
struct ExtendParams : DecodeParams {
  const int32_t *row_start;  // [batch + 1], or null: row b is sequence b's
  int32_t max_rows, rows;    // bound on a sequence's rows; rows of q
  long q_rs, q_hs;           // strides of q between rows and heads, elements
  // warp-MMA kernel: chunks that a change of units counts as in its CTAs'
  // equal shares
  int32_t gap;
  // tcgen05 kernel: pairs of a row block, and chunks of it that one CTA (or
  // pair of CTAs) takes at most
  int32_t block_rows, chunks_per_split;
};

// Rotation of q and k (write false), or the cache write of k and v with the
// optional rotation of q and k (write true).
cudaError_t launch_rows(const RowsParams &p, bool write, int sms,
                        cudaStream_t s);
// Whether one key head's rotation fits in a CTA's shared memory.
bool rows_fit(int d, int half);
// Cached rows as bf16 into k_out and v_out.
cudaError_t launch_read(const RowsParams &p, int sms, cudaStream_t s);
// kvd_gqa_extend, at most kFewPairs (row, head) pairs a kv head: warp-level
// MMAs over units of `hp` kv heads, in chunks of `chunk` positions, `tiles`
// tiles of 8 pairs.
//
// A change of units (kUnitGap): its queries' loads and its outputs take 3 to 5
// us, a chunk about 1.1. (A pass of 32 sequences of 8 kv heads in a graph: 51.5
// us with 0, 50.1 with 3, 49.0 with 4, 49.5 with 6; of 4 kv heads of 16 pairs
// over 18,400 positions: 98.9, 93.9, 93.8, 94.0.) Shares of a few chunks are
// cut evenly.
constexpr int kFewPairs = 16;
constexpr int kUnitGap = 4;
struct FewPlan {
  int hp, chunk, tiles;
};
FewPlan extend_few_plan(int n_kv, int block_size, int pairs, long batch,
                        int max_seq_len, int sms);
cudaError_t launch_extend_few(const ExtendParams &p, const FewPlan &f,
                              cudaStream_t s);
// kvd_gqa_extend otherwise, on tcgen05: blocks of block_rows (row, head)
// pairs of a kv head -- kExtendRows a CTA, 2 kExtendRows a pair of CTAs --
// against chunks of kExtendChunk positions, a block's in equal parts of at
// most chunks_per_split (0: one part; else partials [split][rows][n_h] and a
// merge launch). `blocks`: a bound on the row blocks of the batch, `splits`
// on a block's parts.
constexpr int kExtendRows = 256;
constexpr int kExtendChunk = 128;
cudaError_t launch_extend_tc(const ExtendParams &p, int blocks, int splits,
                             cudaStream_t s);

}  // namespace kvd
