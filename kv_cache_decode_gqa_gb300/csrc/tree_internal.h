// Interface between the C ABI layer (api.cu) and the kernels of kvd_tree.h:
// parameter structs and launcher functions.
#pragma once

#include "prompt_internal.h"

namespace kvd {

constexpr int kTreeNodes = 256;  // KVD_TREE_NODES


struct TreePlanParams {
  const int32_t *parents;  // [rows]
  const int32_t *start;    // [batch]
  const int32_t *row_start;
  uint32_t *masks;     // [rows][words]
  int32_t *positions;  // [rows] or null
  int32_t batch, rows, max_rows, words, window;
  int *err;
};

// kvd_gqa_tree (masks set) and kvd_gqa_cross (masks null). The ExtendParams
// fields it uses keep their meaning; n_splits are the CTAs, block_rows the
// pairs that a partial result has room for.
struct AttendParams : ExtendParams {
  const uint32_t *masks;     // [rows][words]: nodes a row sees
  const int32_t *positions;  // [rows], with a window
  int32_t words;
};

// kvd_kv_keep: up to kKeepCaches caches of one shape a launch.
constexpr int kKeepCaches = 96;
struct KeepParams {
  uint8_t *data[2 * kKeepCaches];  // K (and V) of each cache
  const int32_t *block_table, *start, *path, *n_keep;
  int32_t tensors, row, n_kv;  // entries of data, bytes of a row
  int32_t batch, max_blocks, block_size, num_blocks, width;
  int *err;
};

cudaError_t launch_tree_plan(const TreePlanParams &p, cudaStream_t s);
// The CTAs of a call (at most `ctas`), with equal shares of its chunks, and
// their partial results: two a CTA, of `pairs` (row, head) pairs each.
struct AttendPlan {
  int ctas = 1, pairs = 0, gap = 0, whole_units = 0;
  size_t ws_o_bytes = 0, ws_bytes = 0;
};
AttendPlan attend_plan(int n_kv, int g, int d, int batch, int rows,
                       int max_rows, int max_seq_len, int ctas);
cudaError_t launch_attend(const AttendParams &p, cudaStream_t s);
cudaError_t launch_keep(const KeepParams &p, cudaStream_t s);

}  // namespace kvd
