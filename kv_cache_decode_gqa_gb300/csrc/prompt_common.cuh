// Device helpers shared by the kernels of the prompt path.
#pragma once

#include "kvd_common.cuh"
#include "prompt_internal.h"
#include "stream_k.cuh"

namespace kvd {

// One arrival on the mbarrier at `addr` in another CTA of the cluster (or this
// one, from cluster_saddr) that orders no memory: for arrivals that publish
// tensor memory, whose accesses tcgen05.wait and tcgen05.fence order with any
// synchronisation of the threads. mbar_arrive_remote is for shared memory.
__device__ __forceinline__ void mbar_arrive_remote_relaxed(uint32_t addr) {
  asm volatile(
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr)
      : "memory");
}

// mbar_test_wait and mbar_wait; CLUSTER: with acquire semantics at cluster
// scope, for barriers that other CTAs of the cluster arrive on.
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_test_scope(uint64_t *bar,
                                                uint32_t parity) {
  if constexpr (!CLUSTER) return mbar_test_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;"
      "\n\tselp.u32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_wait_scope(uint64_t *bar,
                                                uint32_t parity) {
  if constexpr (!CLUSTER) return mbar_wait(bar, parity);
  return mbar_test_scope<true>(bar, parity) || mbar_wait_cluster(bar, parity);
}

// The eight E2M1 codes of a word (first code in the low nibble) to four f16
// pairs, exact. The unpacked bytes let the conversion pick its byte itself:
// 41 pairs a cycle and SM against 20 with a shift before each conversion
// (measured with 16 warps, one multiply a pair).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Product of two f16 pairs, each rounded to nearest even.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Exponent field of the power of two that takes a query row whose largest
// bf16 magnitude has bits `amax` into [2^14, 2^15), where f16 holds it (1
// for a row with an infinity or NaN, which then shows in its outputs).
__device__ __forceinline__ int row_exponent(uint32_t amax) {
  const int e = max((int)(amax >> 7), 1);
  return e == 255 ? 127 : min(268 - e, 254);
}

// ---------------------------------------------------------------------------
// sequences with several new rows (kvd_gqa_extend)
// ---------------------------------------------------------------------------
// A row list is followed up to its first descent: the sequences before it
// hold disjoint rows whatever the entries are, those from there on could hold
// another's and are taken to have none.

// New rows of sequence b, which lies before the first descent; 0 where its
// own entries do not fit the call.
__device__ __forceinline__ int seq_rows(const ExtendParams &p, int b) {
  if (!p.row_start) return 1;
  const int r0 = p.row_start[b], r1 = p.row_start[b + 1];
  const bool bad = (r0 < 0) | (r1 < r0) | (r1 > p.rows) |
                   ((long)r1 - r0 > p.max_rows);
  return bad ? 0 : r1 - r0;
}

__device__ __forceinline__ bool descends(const ExtendParams &p, int b) {
  return p.row_start && p.row_start[b + 1] < p.row_start[b];
}

// The first sequence whose entries descend (the batch if none do), by all
// threads of the block through the shared word `at`. Lists that descend are
// the exception: kernels look for any descent on the way (descends) and come
// here when there is one.
__device__ __forceinline__ int first_descent(const ExtendParams &p, int *at) {
  if (threadIdx.x == 0) *at = p.batch;
  __syncthreads();
  for (int b = threadIdx.x; b < p.batch; b += blockDim.x)
    if (descends(p, b)) atomicMin(at, b);
  __syncthreads();
  return *at;
}

// First position that the window of a row at position `pos` (negative: a row
// before the first position) reaches, or some value below 0. Any window fits.
__device__ __forceinline__ int window_lo(const ExtendParams &p, int pos) {
  return max(pos + 1, 0) - p.window;
}

// First position the rows of sequence b (before the first descent) attend to
// (its visible length is T): the first row's window reaches lowest. A sequence
// without rows attends to nothing.
__device__ __forceinline__ int rows_lo(const ExtendParams &p, int b, int T) {
  const int n = seq_rows(p, b);
  if (n == 0) return T;
  int lo = p.win_start ? p.win_start[b] : 0;
  if (p.window > 0) lo = max(lo, window_lo(p, T - n));
  return min(max(lo, 0), T);
}

// Position of the first row of sequence b's first chunk.
__device__ __forceinline__ int rows_first(const ExtendParams &p, int b, int T,
                                          int chunk) {
  const int lo = rows_lo(p, b, T);
  return lo - lo % chunk;
}

// build_partition (stream_k.cuh) for these sequences: `units` units each of
// the chunks of `chunk` positions that the sequence's rows see and of `gap`
// empty ones behind them, which stand for what a change of units costs the
// CTA that makes it. Sequences from the list's first descent, which
// *list_end receives, have no chunks. Every thread of the block calls it; it
// ends with a barrier.
template <int NB>
__device__ __forceinline__ void build_rows_partition(WorkPartitionT<NB> &wp,
                                                     const ExtendParams &p,
                                                     int *len_error,
                                                     int *list_end, int chunk,
                                                     int units, int gap) {
  const int tid = threadIdx.x, nthreads = blockDim.x;
  __shared__ int warp_tot[32];
  // a run of consecutive sequences a thread, then a scan over the threads
  const int per = (p.batch + nthreads - 1) / nthreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  int local = 0;
  bool broken = false;
  for (int b = b0; b < b1; ++b) {
    int T = p.seq_lens[b];
    if (T > p.max_seq_len) {
      *len_error = 1;
      T = p.max_seq_len;
    }
    T = max(T, 0);
    const int lo = rows_lo(p, b, T);
    const int rows = lo < T ? T - (lo - lo % chunk) : 0;
    wp.len[b] = T;
    wp.nch[b] = rows > 0 ? (rows + chunk - 1) / chunk + gap : 0;
    local += wp.nch[b] * units;
    broken |= descends(p, b);
  }
  const int lane = tid & 31, warp = tid >> 5, nwarps = (nthreads + 31) >> 5;
  int x = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_tot[warp] = x;
  const int any_broken = __syncthreads_or(broken);
  int before = 0, total = 0;
  for (int w = 0; w < nwarps; ++w) {
    if (w < warp) before += warp_tot[w];
    total += warp_tot[w];
  }
  int excl = before + x - local;
  for (int b = b0; b < b1; ++b) {
    wp.pre[b] = excl;
    excl += wp.nch[b] * units;
  }
  if (tid == 0) {
    wp.units = units;
    wp.total = total;
    wp.pre[p.batch] = total;
    *list_end = p.batch;
  }
  __syncthreads();
  if (any_broken) {
    const int end = first_descent(p, list_end);
    if (tid == 0) {
      int at = 0;
      for (int b = 0; b < p.batch; ++b) {
        if (b >= end) wp.nch[b] = 0;
        wp.pre[b] = at;
        at += wp.nch[b] * units;
      }
      wp.total = wp.pre[p.batch] = at;
    }
    __syncthreads();
  }
}

}  // namespace kvd
