// Attention of several rows a sequence that is not causal (kvd_gqa_tree,
// kvd_gqa_cross): one warp a (row, query head), its lanes over the channels,
// the running maximum and sum of a softmax in fp32.
#include <cmath>

#include "prompt_common.cuh"
#include "tree_internal.h"

namespace kvd {
namespace {

constexpr int kAttendThreads = 256;

// This lane's channels [E lane, E lane + E) of a cached row.
template <int DT, int D>
__device__ __forceinline__ void load_channels(const uint8_t *cache, long row,
                                              int lane, float (&x)[D / 32]) {
  constexpr int E = D / 32;
  const uint8_t *src = cache + row * row_bytes(D, DT);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lane * E + e;
    if constexpr (DT == DT_BF16) {
      x[e] = __uint_as_float(
          (uint32_t)reinterpret_cast<const uint16_t *>(src)[c] << 16);
    } else if constexpr (DT == DT_FP8) {
      x[e] = f16lo(e4m3x2_to_f16x2(src[c]));
    } else {
      const uint32_t codes = src[c / 2];
      const float s = f16lo(e4m3x2_to_f16x2(src[D / 2 + c / 16]));
      const uint32_t y = e2m1x2_to_f16x2(codes);
      x[e] = (c & 1 ? f16hi(y) : f16lo(y)) * s;
    }
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kAttendThreads)
    attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int E = D / 32;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long item =
      (long)blockIdx.x * (kAttendThreads / 32) + (threadIdx.x >> 5);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    bool down = false;
    for (int b = 0; b < p.batch; ++b) {
      down |= descends(p, b);
      const int n = down ? 0 : seq_rows(p, b);
      if (p.row_start && n == 0 && p.row_start[b] != p.row_start[b + 1])
        report(p.err, DEVERR_LEN);
      if (p.seq_lens[b] > p.max_seq_len ||
          (p.masks && min(max(p.seq_lens[b], 0), p.max_seq_len) < n))
        report(p.err, DEVERR_LEN);
    }
  }
  if (item >= (long)p.rows * p.n_h) return;
  const int row = (int)(item / p.n_h), h = (int)(item % p.n_h);
  int b = 0, r0 = 0;
  for (;; ++b) {
    if (b == p.batch || descends(p, b)) return;
    const int n = seq_rows(p, b);
    r0 = p.row_start ? p.row_start[b] : b;
    if (row >= r0 && row < r0 + n) break;
  }
  const int T = min(max(p.seq_lens[b], 0), p.max_seq_len);
  const int ctx = p.masks ? T - seq_rows(p, b) : T;
  if (ctx < 0) return;
  int lo = p.win_start ? max(p.win_start[b], 0) : 0;
  if (p.masks && p.window > 0)
    lo = max(lo, max(p.positions[row], -1) + 1 - p.window);
  const int G = p.n_h / p.n_kv, kvh = h / G;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float(
        (uint32_t)p.q[row * p.q_rs + h * p.q_hs + lane * E + e] << 16);
    o[e] = 0.f;
  }
  const float scale =
      p.scale_log2 * (DT == DT_FP8 ? p.k_scale[kvh] : 1.f);
  for (int pos = min(lo, ctx); pos < T; ++pos) {
    if (pos >= ctx) {
      const int j = pos - ctx;
      if (!(p.masks[(long)row * p.words + j / 32] >> (j & 31) & 1)) continue;
    }
    int blk = p.block_table[(long)b * p.max_blocks + pos / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      report(p.err, DEVERR_BLOCK);
      blk = 0;
    }
    const long at =
        ((long)blk * p.n_kv + kvh) * p.block_size + pos % p.block_size;
    float x[E], s = 0.f;
    load_channels<DT, D>(p.k, at, lane, x);
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], x[e], s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= scale;
    const float top = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : exp2f(m - top);
    const float w = top == -INFINITY ? 0.f : exp2f(s - top);
    m = top;
    l = fmaf(l, f, w);
    load_channels<DT, D>(p.v, at, lane, x);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(w, x[e], o[e] * f);
  }
  const float inv =
      l == 0.f ? 0.f : (DT == DT_FP8 ? p.v_scale[kvh] : 1.f) / l;
#pragma unroll
  for (int e = 0; e < E; ++e) p.out[item * D + lane * E + e] = f2bf(o[e] * inv);
  if (lane == 0 && p.lse)
    p.lse[item] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int DT, int D>
cudaError_t launch_t(const AttendParams &p, cudaStream_t s) {
  const long per = kAttendThreads / 32;
  const long items = (long)p.rows * p.n_h;
  return launch_pdl(attend_kernel<DT, D>,
                    dim3((unsigned)((items + per - 1) / per)),
                    dim3(kAttendThreads), 0, s, 1, p);
}

}  // namespace

cudaError_t launch_attend(const AttendParams &p, cudaStream_t s) {
  if (p.dtype == DT_MXFP4) return launch_t<DT_MXFP4, 128>(p, s);
  if (p.dtype == DT_FP8)
    return p.dk == 128 ? launch_t<DT_FP8, 128>(p, s)
                       : launch_t<DT_FP8, 64>(p, s);
  return p.dk == 128 ? launch_t<DT_BF16, 128>(p, s)
                     : launch_t<DT_BF16, 64>(p, s);
}

}  // namespace kvd
