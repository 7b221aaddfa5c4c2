// Trees of drafted tokens: their plan (kvd_tree_plan) and the move of their
// accepted rows (kvd_kv_keep).
#include "kvd_common.cuh"
#include "tree_internal.h"

namespace kvd {
namespace {

constexpr int kPlanThreads = kTreeNodes;

// One CTA a sequence, one thread a node: the thread walks up the parents,
// which lie in shared memory, and sets a bit of its mask a step. A walk is as
// long as the node is deep, some ten steps for a drafted tree and 256 for a
// chain of that many. Latency bounds it: a launch, two dependent loads, the
// walk and the stores (2.9 us for one tree of 16 nodes, 5.7 us for 256 trees of
// 117 on average, in a graph; the bytes would take 0.2).
__global__ void __launch_bounds__(kPlanThreads)
    tree_plan_kernel(const __grid_constant__ TreePlanParams p) {
  __shared__ int16_t up[kTreeNodes];
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.x, i = threadIdx.x;
  // a descent of the list at or before this sequence
  bool down = false;
  for (int j = i; j <= b; j += kPlanThreads)
    down |= p.row_start[j + 1] < p.row_start[j];
  const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
  const bool fits = r0 >= 0 && r1 >= r0 && r1 <= p.rows &&
                    (long)r1 - r0 <= p.max_rows;
  if (__syncthreads_or(down) || !fits) {
    if (i == 0 && r0 != r1) report(p.err, DEVERR_LEN);
    return;
  }
  const int n = r1 - r0;
  if (i < n) {
    int a = p.parents[r0 + i];
    if (a < -1 || a >= i) {
      report(p.err, DEVERR_INDEX);
      a = -1;
    }
    up[i] = (int16_t)a;
  }
  __syncthreads();
  if (i >= n) return;
  constexpr int W = kTreeNodes / 32;
  uint32_t m[W];
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] = 0;
  int depth = 0;
  for (int a = i; a >= 0; a = up[a], ++depth) {
    if (p.window == 0 || depth < p.window) {
#pragma unroll
      for (int w = 0; w < W; ++w)
        if (a >> 5 == w) m[w] |= 1u << (a & 31);
    }
  }
  const long row = r0 + i;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < p.words) p.masks[row * p.words + w] = m[w];
  if (p.positions)
    p.positions[row] = (int)((uint32_t)p.start[b] + (uint32_t)(depth - 1));
}

constexpr int kKeepThreads = 256;

// A thread moves one piece of 16 bytes (8 where the rows are multiples of 8
// only, MXFP4's) of every accepted row of a (cache tensor, sequence, head),
// eight rows' loads in flight: with an ascending path from 0 up, row j's source path[j] >= j, so
// that no store of an earlier row reaches a later row's source when rows are
// taken in order. All layers go in one launch, for which the launch and three
// dependent loads (path, block table, rows) take most of the time: 3.7 us for
// one sequence in 32 layers, 5.7 us for 16 sequences in 80 (21 MB: 3.7 TB/s of
// scattered rows of 128 bytes), in a graph. (Pieces of 8 bytes for every type:
// 7.9 us, and with divisions of 64 bits 8.7.)
template <class Piece>
__global__ void __launch_bounds__(kKeepThreads)
    keep_kernel(const __grid_constant__ KeepParams p) {
  __shared__ long at[kTreeNodes], to[kTreeNodes];  // bytes, of head 0
  // (no early trigger: the next launch starts when the rows are moved, so that
  // a decode call behind that one may declare its older rows final)
  pdl_wait();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int n = p.n_keep[b];
  const bool first = blockIdx.x == 0;
  if (n < 0 || n > p.width) {
    if (first && tid == 0) report(p.err, DEVERR_LEN);
    return;
  }
  int bad = 0;
  const int32_t *path = p.path + (long)b * p.width;
  auto row_of = [&](long pos) {
    if (pos < 0 || pos >= (long)p.max_blocks * p.block_size) {
      bad |= DEVERR_POS;
      return 0L;
    }
    // (a sum of two int32: below 2^32, and a division of 32 bits)
    const uint32_t x = (uint32_t)pos, bs = (uint32_t)p.block_size;
    const uint32_t e = x / bs;
    const int blk = p.block_table[(long)b * p.max_blocks + e];
    if (blk < 0 || blk >= p.num_blocks) {
      bad |= DEVERR_BLOCK;
      return 0L;
    }
    return ((long)blk * p.n_kv * p.block_size + (x - e * bs)) * p.row;
  };
  if (tid < n) {
    const int x = path[tid];
    if (x < 0 || (tid > 0 && path[tid - 1] >= x)) bad |= DEVERR_INDEX;
    at[tid] = row_of((long)p.start[b] + x);
    to[tid] = row_of((long)p.start[b] + tid);
  }
  if (__syncthreads_or(bad)) {
    if (first && bad) report(p.err, bad);
    return;
  }
  const int pieces = p.row / (int)sizeof(Piece);
  // 32 bits where the values have them: a fraction of the instructions
  auto div = [](long a, int b) {
    return a >> 32 ? a / b : (long)((uint32_t)a / (uint32_t)b);
  };
  const long items = (long)p.tensors * p.n_kv * pieces;
  for (long x = (long)blockIdx.x * kKeepThreads + tid; x < items;
       x += (long)gridDim.x * kKeepThreads) {
    const long th = div(x, pieces);
    const int c = (int)(x - th * pieces);
    const long t = div(th, p.n_kv);
    uint8_t *base = p.data[t] + (th - t * p.n_kv) * p.block_size * p.row +
                    c * (int)sizeof(Piece);
    for (int j0 = 0; j0 < n; j0 += 8) {
      Piece v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < n)
          v[j] = *reinterpret_cast<const Piece *>(base + at[j0 + j]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < n && at[j0 + j] != to[j0 + j])
          *reinterpret_cast<Piece *>(base + to[j0 + j]) = v[j];
    }
  }
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams &p, cudaStream_t s) {
  return launch_pdl(tree_plan_kernel, dim3(p.batch), dim3(kPlanThreads), 0, s,
                    1, p);
}

cudaError_t launch_keep(const KeepParams &p, cudaStream_t s) {
  const bool wide = p.row % 16 == 0;
  const long items = (long)p.tensors * p.n_kv * (p.row / (wide ? 16 : 8));
  const long blocks = (items + kKeepThreads - 1) / kKeepThreads;
  return launch_pdl(wide ? keep_kernel<uint4> : keep_kernel<uint2>,
                    dim3((unsigned)(blocks < 4096 ? blocks : 4096), p.batch),
                    dim3(kKeepThreads), 0, s, 1, p);
}

}  // namespace kvd
