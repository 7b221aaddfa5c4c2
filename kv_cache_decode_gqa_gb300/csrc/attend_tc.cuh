// Attention of several rows a sequence that is not causal, on the
// 5th-generation tensor cores (kvd_gqa_tree, kvd_gqa_cross).
//
// The (row, head) pairs of a kv head are numbered row-major, pair f = row *
// G + head, so any group size G fills the MMA's M. A unit is a block of up to
// 256 pairs -- two M = 128 tiles -- of one sequence and kv head against all
// the positions that its sequence attends to, in chunks of 128:
//   S = Q K^T   (A = Q in shared memory, B = K chunk, K-major)
//   O += P V    (A = P in tensor memory, over S; B = V chunk, MN-major)
// A tile's S lies in two buffers of 64 positions: while the softmax (a thread
// a pair) turns one into P, the tensor core does PV of the other and the
// scores that follow it. A unit of at most 128 pairs has one tile; then both
// halves work for it, on even and odd chunks, and their states are merged at
// its end. The masks of a tree touch the chunks that hold its nodes only: 32
// columns at a time, a word of bits shifted to the chunk's first position.
//
// The work of a call is the list of all its units' chunks. A persistent launch
// with one CTA per SM takes equal shares of it; units that two shares cut leave
// partial results, which a second launch merges (attend.cu).
//
// bf16 caches feed the MMAs as they are (bf16 products, exact in fp32), rows
// copied by swizzled TMA boxes; rows of fp8 and MXFP4 caches come raw, by bulk
// copies, and eight warps widen them to f16 (exact: 4 and 6 significand bits;
// E4M3's per-head scales go into the scores' and the outputs' factors).
// Rounded to 16 bits are the probabilities -- to bf16 beside bf16 values, as
// the MMA wants one type for both operands: half a step, 2^-9 to 2^-8 of each,
// the size of the bf16 output's own rounding (an error of 0.0023 of the result
// against 0.0017 for a plain fp32 computation rounded once); to f16 beside f16,
// 2^-11 -- and, for f16, queries scaled by a power of two a (row, head), which
// is exact but for elements 2^-29 of the largest. Scores, references and sums
// are fp32. The reference of a pair moves only when a score passes it by 2^8
// (f16: from 2^7 below the maximum, so that P stays below 2^15 and drops only
// what is 2^-32 of the largest); O is then rescaled in tensor memory.
//
// What bounds it: with many pairs the products, 512 cycles an M = N = K = 128
// one (scores of 64 positions take half as long again as they should, 48
// cycles a step of K = 16 against 32: the operands of both come from shared
// memory, 6 KB a step), and in practice the chain from a product's end over
// the softmax to the next product, about 3,100 cycles a chunk of two tiles
// against 2,576 for its products; with few, HBM, as long as that chain keeps
// up (1,850 cycles a chunk of one tile, K and V of which take 2,900 at HBM's
// rate). Measured (us, calls in a graph): 2,011 rows over 20,011 positions, 64
// heads of 8 kv heads, bf16, 840 and 881 on two GPUs (1,570 and 1,497 TFLOP/s, 81
// and 77% of cuBLAS's rate); trees of 500 nodes in 16 sequences over 9,200
// positions (620 MB) 185; of 250 nodes in 32 sequences over 4,600 positions of an
// fp8 cache (310 MB) 102; of 480 nodes in 8 sequences over 18,400 positions of an
// MXFP4 cache 251; one tree of 16 nodes over 4,000 positions 21.
//
// Measured and not kept (the first of these cases, us): two threads a pair and
// step, of 32 columns each, 1,060 against 1,017 then (more warps to issue for,
// a barrier a step); V through the load path (cp.async by four warps) 902
// against 882; pairs of CTAs (cta_group::2, M = 256, half of the tiles each)
// 1,003, trees of 500 nodes 265, MXFP4 299; two-tile chunks weighted 3 to 2 in
// the shares 970 (the wider arithmetic slowed every role). What was: MMA
// operands in uniform registers (1,198 to 1,050), no register spills (what
// local memory holds comes from L2 beside this much shared memory: 1,810 to
// 1,198), queries loaded in whole lines and outputs stored 32 bytes at a time
// (1,017 to 849).
#pragma once

#include <algorithm>
#include <climits>
#include <cmath>

#include "prompt_common.cuh"
#include "tcgen05_pair.cuh"
#include "tmap.h"
#include "tree_internal.h"

namespace kvd {

struct TcParams {
  AttendParams p;
  // bf16 caches: [which][column half][row][64 columns], of K and V the one that
  // lies first first; or one map each where they lie further apart than a map's
  // strides reach
  CUtensorMap map[2];
  int which[2];  // K's and V's
  int far;       // whether V has a map of its own
  int box;  // rows of its boxes: 1 .. 64, a power of two
};

namespace {

constexpr int kM = 128;         // pairs per tile
constexpr int kUnit = 256;      // pairs per unit, at most
constexpr int kN = 128;         // positions per chunk
constexpr int kS = 64;          // positions per product (half a chunk)
constexpr int kSoftBar = 1;     // named barrier of the softmax warps
constexpr int kSeqs = 12;       // sequences of a CTA's range kept at hand

// DT, D: the cache's type and head width. QS: slots for tiles of queries (1:
// every unit of the launch has one tile).
template <int DT, int D, int QS>
struct ACfg {
  static constexpr bool WIDEN = DT != DT_BF16;
  static constexpr int TILE = 128 * D * 2;    // 128 rows of 16 bits
  static constexpr int HALF = TILE / 2;       // 64 positions of a chunk
  static constexpr int COLS = 64 * 128;       // 64 rows x 64 columns
  static constexpr int RAW = kN * row_bytes(D, DT);  // cached rows of a chunk
  // warps: 0-7 softmax; then four of queries (WIDEN: and K), (WIDEN) four of V,
  // copies of K, (bf16) copies of V, two of MMA issue, (WIDEN) copies of V
  static constexpr int SOFT = 8;
  static constexpr int kLoad = SOFT + (WIDEN ? 8 : 4);
  static constexpr int kLoadV = kLoad + (WIDEN ? 3 : 1);
  static constexpr int kMma = kLoad + (WIDEN ? 1 : 2);
  static constexpr int THREADS = (SOFT + (WIDEN ? 12 : 8)) * 32;
  // a ring of K tiles, one of V tiles, then (WIDEN) raw K and V rows
  static constexpr int SCALES = WIDEN ? QS : 0;
  static constexpr int FIXED = (2 + SCALES) * kM * 4 + 896;
  static constexpr int ROOM = 227 * 1024 - FIXED - QS * TILE;
  static constexpr int NS =
      WIDEN ? 4 : (ROOM / TILE > 12 ? 12 : ROOM / TILE);
  static constexpr int KS = NS / 2, VS = NS - KS;
  // slots and phases of the tiles of chunk g of a CTA's range
  __device__ static __forceinline__ int k_slot(int g) { return g % KS; }
  __device__ static __forceinline__ int v_slot(int g) { return KS + g % VS; }
  __device__ static __forceinline__ uint32_t k_par(int g) {
    return g / KS & 1;
  }
  __device__ static __forceinline__ uint32_t v_par(int g) {
    return g / VS & 1;
  }
  static constexpr int NR_FIT = WIDEN ? (ROOM - NS * TILE) / (RAW + 16) : 0;
  static constexpr int NR = NR_FIT > 12 ? 12 : NR_FIT & ~1;
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = QS * TILE;
  static constexpr int RAW_OFF = KV_OFF + NS * TILE;
  static constexpr int F_OFF = RAW_OFF + NR * RAW;  // float [2][128]
  static constexpr int SL_OFF = F_OFF + 2 * kM * 4;  // float [SCALES][128]
  static constexpr int BAR_OFF = SL_OFF + SCALES * kM * 4;
  static constexpr int BARS = 3 * NS + 2 * NR + 2 * QS + 13;
  static constexpr int FLAG_OFF = BAR_OFF + BARS * 8;
  static constexpr int SEQ_OFF = FLAG_OFF + 32;  // Seq [kSeqs]
  static constexpr int SEEN_OFF = SEQ_OFF + kSeqs * 32;  // uint32 [NR][4]
  static constexpr int SMEM = SEEN_OFF + NR * 16;
  static_assert(NS >= 4 && (!WIDEN || NR >= 2) && SMEM <= 227 * 1024,
                "shared memory");
  static_assert(RAW % 128 == 0 && FLAG_OFF % 8 == 0, "alignment");
};

// 16-byte piece c (0..7) of row r (0..63) in a 128-byte-swizzled 64-column
// tile.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// Packed pairs of fp32 values, one instruction for both.
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b,
                                              uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest of three, NaN only if all are.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ int uniform(int x) {
  return __shfl_sync(0xffffffffu, x, 0);
}

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, int x,
                                            int y, int z, int w,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::"
      "complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// 8 columns of this thread's lane of tensor memory, waited for, and back.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, "
      "[%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr,
                                         const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, "
      "%7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7])
      : "memory");
}

// 32 bytes at once, on a 32-byte boundary.
__device__ __forceinline__ void st_global_v8(float *dst, const float *y) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                   dst),
               "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]),
               "f"(y[5]), "f"(y[6]), "f"(y[7])
               : "memory");
}

// ---------------------------------------------------------------------------
// the work: every chunk of every unit, in the order (sequence, kv head, block
// of pairs, chunk); the CTAs take equal consecutive ranges
// ---------------------------------------------------------------------------
// What a sequence's units are computed from.
struct Seq {
  int r0, n;    // its rows (n = 0: skipped, or none)
  int T, ctx;   // positions, and those before the tree (cross: all)
  int lo;       // first position that a row attends to
  int nch;      // chunks
  int blocks;   // blocks of pairs
  int pad;
  __device__ __forceinline__ int c0() const { return lo / kN; }
};
static_assert(sizeof(Seq) == 32, "shared memory");

__device__ __forceinline__ Seq seq_at(const AttendParams &p, int b, int G) {
  Seq q;
  q.r0 = p.row_start ? p.row_start[b] : b;
  q.n = seq_rows(p, b);
  q.T = min(max(p.seq_lens[b], 0), p.max_seq_len);
  q.ctx = q.T;
  q.lo = p.win_start ? max(p.win_start[b], 0) : 0;
  if (p.masks) {
    q.ctx = q.T - q.n;
    if (q.ctx < 0) q.n = 0;
    if (p.window > 0) q.lo = max(q.lo, max(q.ctx, 0) - (p.window - 1));
    q.lo = min(q.lo, max(q.ctx, 0));
  }
  q.nch = q.n > 0 && q.lo < q.T ? (q.T + kN - 1) / kN - q.c0() : 0;
  q.blocks = (int)(((long)q.n * G + kUnit - 1) / kUnit);
  return q;
}

// What a unit counts as in the shares: its chunks and p.gap empty ones behind
// them, which stand for what a change of units costs the CTA that makes it; or
// 1, where units are not cut.
__device__ __forceinline__ int unit_len(const AttendParams &p, const Seq &q) {
  return p.whole_units ? 1 : q.nch + p.gap;
}
__device__ __forceinline__ long seq_chunks(const AttendParams &p,
                                           const Seq &q) {
  return q.nch == 0 ? 0 : (long)p.n_kv * q.blocks * unit_len(p, q);
}

// Exclusive prefix sums of the sequences' chunks over the block's threads:
// thread t has the (at most SPT) sequences [t per, t per + per), per =
// ceil(batch / blockDim), and keeps them in `q`; those from the list's first
// descent on, which `end` receives, have no chunks. `scratch`: int64 [33].
// Ends with a barrier.
template <int SPT>
__device__ __forceinline__ void scan_work(const AttendParams &p, int G,
                                          long *scratch, Seq (&q)[SPT],
                                          long &before, long &total,
                                          int &end) {
  const int tid = threadIdx.x, nt = blockDim.x;
  const int lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int per = (p.batch + nt - 1) / nt, b0 = tid * per;
  bool broken = false;
#pragma unroll
  for (int j = 0; j < SPT; ++j) {
    q[j].nch = q[j].n = q[j].blocks = 0;
    if (j < per && b0 + j < p.batch) {
      q[j] = seq_at(p, b0 + j, G);
      broken |= descends(p, b0 + j);
    }
  }
  end = p.batch;
  if (__syncthreads_or(broken)) {
    end = first_descent(p, reinterpret_cast<int *>(scratch + 32));
#pragma unroll
    for (int j = 0; j < SPT; ++j)
      if (b0 + j >= end) q[j].nch = q[j].n = q[j].blocks = 0;
  }
  long sum = 0;
#pragma unroll
  for (int j = 0; j < SPT; ++j) sum += seq_chunks(p, q[j]);
  long x = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  long w = lane < nw ? scratch[lane] : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long upto = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  before = (warp > 0 ? upto : 0) + x - sum;
  __syncthreads();
}

// a / b of values that are not negative: 32 bits are faster by a few hundred
// cycles.
__device__ __forceinline__ long div_u(long a, int b) {
  return a >> 32 ? a / b : (long)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ long share_lo(int c, long total, int P) {
  const long each = div_u(total, P);
  return each * c + (total - each * P) * c / P;
}
// The CTA whose share holds chunk x.
__device__ __forceinline__ int share_of(long x, long total, int P) {
  int c = (int)((double)x / (double)total * P);
  c = min(max(c, 0), P - 1);
  while (c > 0 && x < share_lo(c, total, P)) --c;
  while (c < P - 1 && x >= share_lo(c + 1, total, P)) ++c;
  return c;
}

// Where a role is in its CTA's range. A role's loops keep this much only and
// look the rest up (Seg) when a unit begins and ends: what registers cannot
// hold goes to local memory, which beside this much shared memory means L2.
struct Walk {
  int b, unit;  // sequence, unit of it (kv head major, blocks of pairs)
  int k0;       // first chunk of the unit
  long left;    // chunks from here on
};

// A CTA's run of chunks of one unit.
struct Seg {
  Seq q;
  int h;        // kv head
  int f0, np;   // first pair, pairs
  int k0, nch;  // its chunks, [k0, k0 + nch) of q.nch; none in a gap
  bool two;     // two tiles
  __device__ __forceinline__ int c0() const { return q.c0() + k0; }
  __device__ __forceinline__ bool whole() const { return nch == q.nch; }
  // chunks that tile t takes part in, two steps each
  __device__ __forceinline__ int steps(int t) const {
    return two ? 2 * nch : (nch - t + 1) & ~1;
  }
  __device__ __forceinline__ int tiles() const { return two ? 2 : 1; }
};

// Step v of tile t: half v & 1 of this chunk of the segment.
__device__ __forceinline__ int chunk_of(bool two, int t, int v) {
  return two ? v >> 1 : (v & ~1) + t;
}

// Sequence b of the range; `near`: b0 .. b0 + kSeqs - 1.
__device__ __forceinline__ Seq seq_near(const AttendParams &p, int b, int G,
                                        const Seq *near, int b0) {
  return b - b0 < kSeqs ? near[b - b0] : seq_at(p, b, G);
}

__device__ __forceinline__ Seg seg_at(const AttendParams &p, const Walk &w,
                                      int G, const Seq *near, int b0) {
  Seg s;
  s.q = seq_near(p, w.b, G, near, b0);
  s.h = w.unit / s.q.blocks;
  s.f0 = (w.unit - s.h * s.q.blocks) * kUnit;
  s.np = min(s.q.n * G - s.f0, kUnit);
  s.two = s.np > kM;
  s.k0 = w.k0;
  s.nch = p.whole_units ? s.q.nch
                        : (int)min((long)max(s.q.nch - s.k0, 0), w.left);
  return s;
}

// On to the segment after `s`; false at the range's end.
__device__ __forceinline__ bool walk_on(const AttendParams &p, Walk &w,
                                        const Seg &s, int G, const Seq *near,
                                        int b0) {
  w.left -= unit_len(p, s.q) - s.k0;
  if (w.left <= 0) return false;
  w.k0 = 0;
  if (++w.unit == p.n_kv * s.q.blocks) {
    w.unit = 0;
    do ++w.b;
    while (seq_near(p, w.b, G, near, b0).nch == 0);
  }
  return true;
}

// Bits of the 32 positions from p0 on that a row sees: [lo, ctx), and the
// nodes of its mask (`words` words at `mask`, n nodes from position ctx on).
__device__ __forceinline__ uint32_t seen_bits(int p0, int lo, int ctx, int n,
                                              const uint32_t *mask,
                                              int words) {
  const int a = min(max(lo - p0, 0), 32), z = min(max(ctx - p0, 0), 32);
  uint32_t bits = 0;
  if (a < z) bits = (0xffffffffu >> (32 - (z - a))) << a;
  const int j = p0 - ctx;  // the first position's node
  if (mask && j > -32 && j < n) {
    const int w = j >> 5;
    const uint32_t x = w >= 0 ? mask[w] : 0u;
    const uint32_t y = w + 1 < words ? mask[w + 1] : 0u;
    uint32_t m = __funnelshift_r(x, y, j & 31);
    if (n - j < 32) m &= (1u << (n - j)) - 1u;  // nodes from n on
    bits |= m;
  }
  return bits;
}

// What no row of a sequence sees may hold anything, but meets a probability of
// 0 in the product with V, where 0 times NaN would be NaN: such rows of V are
// zeros there. The next two are called by whole warps.
//
// First position of the context that some row of sequence b sees (q.ctx or more:
// none). q.lo, which the work is shared out by, stands for a row at the tree's
// first position.
__device__ __forceinline__ int first_seen(const AttendParams &p, const Seq &q,
                                          int b, int lane) {
  if (!p.masks) return q.lo;
  int lo = p.win_start ? max(p.win_start[b], 0) : 0;
  if (p.window > 0) {
    int pos = INT_MAX;
    for (int i = lane; i < q.n; i += 32)
      pos = min(pos, p.positions[q.r0 + i]);
    pos = __reduce_min_sync(0xffffffffu, pos);
    lo = max(lo, max(pos, q.ctx) - (p.window - 1));
  }
  return lo;
}

// Bits of the 32 positions from p0 on that some row of the sequence sees
// (`first`: first_seen).
__device__ __forceinline__ uint32_t seen_by_some(const AttendParams &p,
                                                 const Seq &q, int first,
                                                 int p0, int lane) {
  if (!p.masks || p0 + 32 <= q.ctx)
    return seen_bits(p0, first, q.ctx, 0, nullptr, 0);
  uint32_t bits = 0;
#pragma unroll 4
  for (int i = lane; i < q.n; i += 32)
    bits |= seen_bits(p0, first, q.ctx, q.n,
                      p.masks + (long)(q.r0 + i) * p.words, p.words);
  return __reduce_or_sync(0xffffffffu, bits);
}

template <int DT, int D, int QS>
__global__ void __launch_bounds__(ACfg<DT, D, QS>::THREADS, 1)
    attend_tc_kernel(const __grid_constant__ TcParams tp) {
  using C = ACfg<DT, D, QS>;
  constexpr bool WIDEN = C::WIDEN;
  constexpr int NS = C::NS, NR = C::NR;
  // log2 units that a reference lies below the maximum, and may lag by: f16
  // probabilities stay below 2^15 and the largest is at least 2^7, so that f16
  // drops only what is 2^-32 of it; bf16 has fp32's range
  constexpr float kHead = WIDEN ? 7.f : 0.f;
  constexpr float kSlack = 8.f;
  // tensor memory: two score buffers of 64 columns a tile, then the outputs
  constexpr uint32_t kColS = 0, kColO = 256;
  const AttendParams &p = tp.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  float *fs = reinterpret_cast<float *>(smem + C::F_OFF);
  float *qsl = reinterpret_cast<float *>(smem + C::SL_OFF);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
  uint64_t *empty = full + NS;
  uint64_t *land = empty + NS;  // bf16: a V tile whose ends are not filled
  uint64_t *rawfull = land + NS;
  uint64_t *rawempty = rawfull + NR;
  uint64_t *qfull = rawempty + NR;
  uint64_t *qempty = qfull + QS;
  uint64_t *sfull = qempty + QS;  // [tile][buffer]
  uint64_t *pfull = sfull + 4;    // [tile][buffer]
  uint64_t *pvdone = pfull + 4;   // [tile]
  uint64_t *odone = pvdone + 2;   // [tile]: a unit's last product
  uint64_t *drain = odone + 2;
  int *flags = reinterpret_cast<int *>(smem + C::FLAG_OFF);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(flags);
  int *s_b = flags + 1;
  long *s_off = reinterpret_cast<long *>(flags + 2);

  Seq *near = reinterpret_cast<Seq *>(smem + C::SEQ_OFF);
  // rows of the raw V slots that some row of the sequence attends to
  uint32_t *seen_v = reinterpret_cast<uint32_t *>(smem + C::SEEN_OFF);

  // (through a shuffle: the compiler then knows the warp's number, and what
  // follows from it, to be the same for its lanes, and keeps the operands of
  // the MMAs in uniform registers)
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const int G = p.n_h / p.n_kv;

  // ---- what needs nothing of the launch before --------------------------
  // the swizzled tiles assume 1 KB atoms (every CTA sees the same layout)
  const bool placed = (smem_u32(smem) & 1023u) == 0;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], WIDEN ? 4 : 1);
      mbar_init(&empty[i], 2);  // both MMA warps
      mbar_init(&land[i], 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(&rawfull[i], 1);
      mbar_init(&rawempty[i], 4);
    }
    for (int i = 0; i < QS; ++i) {
      mbar_init(&qfull[i], WIDEN ? 8 : 4);
      // a commit of either MMA warp (and the softmax warps have the scales)
      mbar_init(&qempty[i], WIDEN ? 2 + C::SOFT : 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
    }
    mbar_init(&pvdone[0], 1);
    mbar_init(&pvdone[1], 1);
    mbar_init(&odone[0], 1);
    mbar_init(&odone[1], 1);
    mbar_init(drain, 2);
    fence_mbar_init();
  }
  if (!WIDEN && (warp == C::kLoad || warp == C::kLoadV) && lane == 0)
    prefetch_tmap(&tp.map[warp == C::kLoadV && tp.far]);
  if (warp == C::kMma) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *s_tmem;
  pdl_wait();
  pdl_trigger();  // after the wait: the merge launch never overlaps this
                  // launch's predecessor
  // ---- this CTA's share ------------------------------------------------
  long lo = 0, hi = 0;
  {
    constexpr int SPT = (kMaxDecodeBatch + C::THREADS - 1) / C::THREADS;
    Seq q[SPT];
    long before, total;
    int end;
    scan_work(p, G, reinterpret_cast<long *>(smem), q, before, total, end);
    const int P = (int)min((long)gridDim.x, total), c = blockIdx.x;
    if (c < P) {
      lo = share_lo(c, total, P);
      hi = share_lo(c + 1, total, P);
    }
    const int per = (p.batch + C::THREADS - 1) / C::THREADS, b0 = tid * per;
    bool zeros = false;  // rows that see nothing, of sequences of this CTA
#pragma unroll
    for (int j = 0; j < SPT; ++j) {
      const int b = b0 + j;
      if (j >= per || b >= p.batch) continue;
      const long n = seq_chunks(p, q[j]);
      if (lo < hi && lo >= before && lo < before + n) {
        *s_b = b;
        *s_off = lo - before;
      }
      before += n;
      zeros |= q[j].n > 0 && q[j].nch == 0 && b % gridDim.x == c;
      if (c == 0) {
        const bool rows = p.row_start && p.row_start[b] != p.row_start[b + 1];
        if ((rows && q[j].n == 0) || p.seq_lens[b] > p.max_seq_len)
          report(p.err, DEVERR_LEN);
      }
    }
    if (__syncthreads_or(zeros)) {
      for (int b = c; b < end; b += gridDim.x) {
        const Seq s = seq_at(p, b, G);
        if (s.n == 0 || s.nch > 0) continue;
        for (long i = tid; i < (long)s.n * p.n_h * (D / 8); i += C::THREADS)
          reinterpret_cast<uint4 *>(p.out + (long)s.r0 * p.n_h * D)[i] =
              make_uint4(0, 0, 0, 0);
        if (p.lse)
          for (long i = tid; i < (long)s.n * p.n_h; i += C::THREADS)
            p.lse[(long)s.r0 * p.n_h + i] = -INFINITY;
      }
    }
    if (lo < hi) {
#pragma unroll
      for (int j = 0; j < SPT; ++j) {
        const int i = b0 + j - *s_b;
        if (j < per && b0 + j < p.batch && i >= 0 && i < kSeqs) near[i] = q[j];
      }
    }
    __syncthreads();
  }
  if (!placed && tid == 0) report(p.err, DEVERR_TIMEOUT);
  if (lo >= hi || !placed) {
    if (warp == C::kMma) tmem_dealloc(tbase, 512);
    return;
  }
  const int b_near = *s_b;
  Walk wk;
  wk.b = b_near;
  wk.unit = (int)div_u(*s_off, unit_len(p, near[0]));
  wk.k0 = (int)(*s_off - (long)wk.unit * unit_len(p, near[0]));
  wk.left = hi - lo;
  auto here = [&]() { return seg_at(p, wk, G, near, b_near); };
  auto next = [&](const Seg &s) {
    return walk_on(p, wk, s, G, near, b_near);
  };
  {
    // a range that begins in a gap; all of it may be one
    const Seg s = here();
    if (s.nch == 0 && !next(s)) {
      if (warp == C::kMma) tmem_dealloc(tbase, 512);
      return;
    }
  }
  // Every wait is bounded. A role whose wait runs out goes on without waiting
  // and without touching what it waited for; the others follow when their own
  // waits run out.
  auto give_up = [&]() {
    if (lane == 0) report(p.err, DEVERR_TIMEOUT);
  };
  auto wait_all = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
  };
  // Uses of the query slots, in order: a unit's tiles one after the other.
  auto q_slot = [&](int use) { return use % QS; };
  auto q_par = [&](int use) { return (uint32_t)(use / QS & 1); };

  // Rows [r0, r0 + ROWS) of a tile of queries by 128 threads: side by side, so
  // that the loads are whole lines, several in flight a thread (WIDEN: scaled
  // into f16).
  constexpr int ROWS = WIDEN ? 64 : 128;
  auto load_queries = [&](const Seg &s, int t, int use, int x, int r0) {
    constexpr int LPR = D / 8, RP = 128 / LPR;  // lanes a row, rows at a time
    constexpr int NF = WIDEN ? 4 : 8;
    const int c = x % LPR;
    int r = r0 + x / LPR;
    int f = s.f0 + t * kM + r, row = s.q.r0 + f / G, g = f % G;
    const int dr = RP / G, dg = RP % G;
    uint8_t *qt = smem + C::Q_OFF + q_slot(use) * C::TILE;
#pragma unroll 1
    for (int i0 = 0; i0 < ROWS / RP; i0 += NF) {
      uint4 w[NF];
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (t * kM + r + i * RP < s.np)
          w[i] = *reinterpret_cast<const uint4 *>(
              p.q + (long)row * p.q_rs + ((long)s.h * G + g) * p.q_hs + c * 8);
        row += dr, g += dg;
        if (g >= G) ++row, g -= G;
      }
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        if constexpr (WIDEN) {
          uint32_t m =
              __vmaxu2(__vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu),
                       __vmaxu2(w[i].z & 0x7fff7fffu, w[i].w & 0x7fff7fffu));
          m = max(m & 0xffffu, m >> 16);
#pragma unroll
          for (int off = 1; off < LPR; off <<= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
          const int e = row_exponent(m);
          const float sc = __uint_as_float((uint32_t)e << 23);
          if (c == 0)
            qsl[q_slot(use) * kM + r] =
                fmaxf(p.scale_log2 * (DT == DT_FP8 ? p.k_scale[s.h] : 1.f) *
                          exp2f((float)(127 - e)),
                      1.17549435e-38f);
          w[i] = make_uint4(
              pack_f16x2(bf16lo(w[i].x) * sc, bf16hi(w[i].x) * sc),
              pack_f16x2(bf16lo(w[i].y) * sc, bf16hi(w[i].y) * sc),
              pack_f16x2(bf16lo(w[i].z) * sc, bf16hi(w[i].z) * sc),
              pack_f16x2(bf16lo(w[i].w) * sc, bf16hi(w[i].w) * sc));
        }
        // 64 rows of 64 columns lie 8 KB apart, columns from 64 on behind all
        // rows
        *reinterpret_cast<uint4 *>(qt + ((c >> 3) * 2 + (r >> 6)) * C::COLS +
                                   sw128(r & 63, c & 7)) = w[i];
        r += RP;
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&qfull[q_slot(use)]);
  };

  if (warp < C::SOFT) {
    // ======================= softmax ======================================
    if constexpr (WIDEN) reg_inc<128>();
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // pair of the tile
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    int use = 0;              // query slots used so far
    int gv = 0, units = 0;    // steps (pairs of them) and units so far
    bool ok = true;
    while (true) {
      // ---- what the steps need -------------------------------------------
      // what the pair sees (one that does not exist: everything, so that its
      // warp masks nothing for it; its query is 0 and nothing of it is stored)
      int vlo = 0, vctx = INT_MAX, row = -1;
      int nv, first, nodes;
      bool two, live;
      {
        const Seg sg = here();
        two = sg.two;
        nv = sg.steps(t);
        first = sg.c0() * kN;
        nodes = sg.q.n;
        const int ri = two ? t * kM + r : r;  // pair of the unit
        live = ri < sg.np;
        if (live) {
          vlo = p.win_start ? max(p.win_start[wk.b], 0) : 0;
          vctx = sg.q.ctx;
          if (p.masks) {
            row = sg.q.r0 + (sg.f0 + ri) / G;
            if (p.window > 0)
              vlo = max(vlo, max(p.positions[row], vctx) - (p.window - 1));
          }
        }
      }
      const bool warp_live = __any_sync(0xffffffffu, live);
      float sl = p.scale_log2;
      if constexpr (WIDEN) {
        // (the other tile's slot is released here too)
        for (int i = 0; i <= (int)two; ++i) {
          if (ok && !wait_all(&qfull[q_slot(use + i)], q_par(use + i))) {
            give_up();
            ok = false;
          }
        }
        const int u = use + (two ? t : 0);
        sl = qsl[q_slot(u) * kM + r];
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&qempty[q_slot(use)]);
          if (two) mbar_arrive(&qempty[q_slot(use + 1)]);
        }
      }
      use += two ? 2 : 1;
      float ref = -INFINITY, l = 0.f;
      for (int v = 0; v < nv; ++v) {
        const int buf = v & 1;
        const int p0 = first + chunk_of(two, t, v) * kN + buf * kS;
        if (ok && !wait_all(&sfull[2 * t + buf], (gv + (v >> 1)) & 1)) {
          give_up();
          ok = false;
        }
        tc_fence_after();
        if (warp_live) {
          uint32_t x[2][32];
          const uint32_t ts = tl + kColS + 128 * t + kS * buf;
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_ld32(ts + 32 * i, x[i]);
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_wait_ld(x[i]);
          // columns that some pair of the warp does not see
          if (__any_sync(0xffffffffu, p0 < vlo || p0 > vctx - kS)) {
            const uint32_t *mask =
                row >= 0 ? p.masks + (long)row * p.words : nullptr;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t bits =
                  live ? seen_bits(p0 + 32 * i, vlo, vctx, nodes, mask,
                                   p.words)
                       : 0xffffffffu;
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(bits >> j & 1)) x[i][j] = 0xff800000u;  // -inf
            }
          }
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t *y = &x[i >> 1][16 * (i & 1)];
            mx[i] = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
#pragma unroll
            for (int j = 2; j < 16; j += 2)
              mx[i] = max3(mx[i], __uint_as_float(y[j]),
                           __uint_as_float(y[j + 1]));
          }
          const float top =
              fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * sl - kHead;
          const bool grow = top > ref + kSlack;  // from -inf: any score
          if (__any_sync(0xffffffffu, grow)) {
            const float al = grow ? ex2(ref - top) : 1.f;
            if (grow) ref = top;
            l *= al;
            if (v > 0) {
              // the tile's last product into O has to be over (this step's
              // scores followed the one before it)
              if (ok && !wait_all(&pvdone[t], (v - 1) & 1)) {
                give_up();
                ok = false;
              }
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < D / 8; ++i) {
                uint32_t o[8];
                const uint32_t to = tl + kColO + D * t + 8 * i;
                tmem_ld8(to, o);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
                tmem_st8(to, o);
              }
            }
          }
          const float mu = ref == -INFINITY ? 0.f : ref;
          const uint64_t mu2 = pack_f32x2(-mu, -mu);
          const uint64_t sl2 = pack_f32x2(sl, sl);
          uint64_t ls[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t pk[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float e0, e1;
              unpack_f32x2(
                  fma_f32x2(pack_f32x2(__uint_as_float(x[i][2 * j]),
                                       __uint_as_float(x[i][2 * j + 1])),
                            sl2, mu2),
                  e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              ls[j & 1] = add_f32x2(ls[j & 1], pack_f32x2(e0, e1));
              pk[j] = WIDEN ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
            }
            // (over the scores of its own pair, which it has read)
            tmem_st16(ts + 16 * i, pk);
          }
          {
            float a0, a1;
            unpack_f32x2(add_f32x2(ls[0], ls[1]), a0, a1);
            l += a0 + a1;
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[2 * t + buf]);
      }
      // ---- epilogue ------------------------------------------------------
      gv += nv >> 1;
      if (nv > 0) {
        if (ok && !wait_all(&odone[t], units & 1)) {
          give_up();
          ok = false;
        }
        ++units;
      }
      tc_fence_after();
      // (looked up again: see Walk)
      asm volatile("" : "+r"(wk.b), "+r"(wk.unit), "+r"(wk.k0));
      const Seg sg = here();
      const int ri = two ? t * kM + r : r, f = sg.f0 + ri;
      // the outputs' factors (of the tile's sums, and of tile 1's in one-tile
      // units) and the log-sum-exp
      float w0, w1 = 0.f, lse = 0.f;
      auto finish = [&](float M, float L) {
        lse = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        return L == 0.f ? 0.f : DT == DT_FP8 ? p.v_scale[sg.h] / L : 1.f / L;
      };
      if (two) {
        w0 = finish(ref, l);
      } else {
        // the two tiles' states of pair r, joined by tile 0's thread
        if (t == 1) fs[r] = ref, fs[kM + r] = l;
        tc_fence_before();
        named_sync(kSoftBar, 256);
        tc_fence_after();
        if (t == 0) {
          const float rb = fs[r], M = fmaxf(ref, rb);
          const float mu = M == -INFINITY ? 0.f : M;
          w0 = ex2(ref - mu);
          w1 = ex2(rb - mu);
          const float inv = finish(M, l * w0 + fs[kM + r] * w1);
          fs[r] = w0 *= inv, fs[kM + r] = w1 *= inv;
        }
        named_sync(kSoftBar, 256);
        w0 = fs[r], w1 = fs[kM + r];
      }
      const bool whole = sg.whole();
      const long at =
          ((long)sg.q.r0 + f / G) * p.n_h + (long)sg.h * G + f % G;
      const long part = ((long)blockIdx.x * 2 + (sg.k0 > 0 ? 0 : 1)) *
                            p.block_rows + ri;
      // two tiles: all columns of the tile's pair, 64 at a time; one: half of
      // them by each tile's thread, 32 at a time of either tile's sums
      const bool second = !two && sg.nch > 1;
      const int col0 = two ? 0 : t * (D / 2), step = two ? 64 : 32;
      const uint32_t to = tl + kColO + (two ? D * t : 0);
      // (a weight of 0 is that of a tile whose pair saw nothing; its sums are
      // NaN beside values that are not finite)
      auto times = [](uint32_t o, float w) {
        return w == 0.f ? 0.f : __uint_as_float(o) * w;
      };
      auto emit = [&](int col, const float (&y)[32]) {
        if (whole) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + at * D + col);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]),
                                pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                pack_bf16x2(y[8 * i + 4], y[8 * i + 5]),
                                pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_global_v8(p.ws_o + part * D + col + 8 * i, y + 8 * i);
        }
      };
      if (warp_live && ok) {
#pragma unroll 1
        for (int g = col0; g < (two ? D : col0 + D / 2); g += step) {
          uint32_t o[2][32];
          tmem_ld32(to + g, o[0]);
          if (two)
            tmem_ld32(to + g + 32, o[1]);
          else
            tmem_ld32(to + D + (second ? g : col0), o[1]);
          tmem_wait_ld(o[0]);
          tmem_wait_ld(o[1]);
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            y[i] = times(o[0][i], w0);
          if (second && w1 != 0.f) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              y[i] = fmaf(__uint_as_float(o[1][i]), w1, y[i]);
          }
          if (live) emit(g, y);
          if (two) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              y[i] = times(o[1][i], w0);
            if (live) emit(g + 32, y);
          }
        }
        if (live && (two || t == 0)) {
          if (!whole)
            p.ws_lse[part] = lse;
          else if (p.lse)
            p.lse[at] = lse;
        }
      }
      tc_fence_before();
      // (the next unit's products into O and its states wait for all reads)
      if (!two) named_sync(kSoftBar, 256);
      if (!next(sg)) break;
    }
  } else if (WIDEN && warp < C::SOFT + 8) {
    // ======================= queries, widening ============================
    if constexpr (WIDEN) {
      reg_dec<72>();
      const int r = tid & 127;  // row of the chunk
      const bool is_v = warp >= C::SOFT + 4;
      int use = 0, gc = 0;
      bool ok = true;
      // K rows are raw units 0, 2, 4, ..., V rows 1, 3, 5, ...
      int rs = is_v, rph = 0;
      Seg sg;
      do {
        sg = here();
        for (int t = 0; t < sg.tiles(); ++t, ++use) {
          if (ok && !wait_all(&qempty[q_slot(use)], q_par(use) ^ 1)) {
            give_up();
            ok = false;
          }
          if (ok) load_queries(sg, t, use, r, 64 * is_v);
        }
        for (int i = 0; ok && i < sg.nch; ++i, ++gc) {
          if (!wait_all(&rawfull[rs], rph)) {
            give_up();
            ok = false;
            break;
          }
          const uint8_t *src =
              smem + C::RAW_OFF + rs * C::RAW + r * row_bytes(D, DT);
          // a row of V that was not copied, or that no pair sees: zeros, so
          // that 0 times it stays 0 (scores of such a row are masked)
          const bool dead =
              is_v && !(seen_v[4 * rs + (r >> 5)] >> lane & 1);
          const int st = is_v ? C::v_slot(gc) : C::k_slot(gc);
          const uint32_t free_par =
              (is_v ? C::v_par(gc) : C::k_par(gc)) ^ 1;
          uint8_t *dst = smem + C::KV_OFF + st * C::TILE + (r >> 6) * C::HALF;
          constexpr int PIECES = D / 16;  // of 16 channels
          auto put = [&](int g, const uint32_t (&y)[8]) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int c = 2 * g + q;
              *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::COLS +
                                         sw128(r & 63, c & 7)) =
                  make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2],
                             y[4 * q + 3]);
            }
          };
          // raw codes to registers, then the slot is free. (The copies into it
          // are of another proxy: without the fence they overtook loads that
          // the threads had issued but not received, once in some hundred
          // calls.)
          auto raw_free = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&rawempty[rs]);
          };
          if constexpr (DT == DT_MXFP4) {
            uint2 w[PIECES];
            uint32_t sw[PIECES / 4];
#pragma unroll
            for (int g = 0; g < PIECES; ++g)
              w[g] = *reinterpret_cast<const uint2 *>(src + 8 * g);
#pragma unroll
            for (int g = 0; g < PIECES / 4; ++g)
              sw[g] =
                  *reinterpret_cast<const uint32_t *>(src + D / 2 + 4 * g);
            if (dead) {
#pragma unroll
              for (int g = 0; g < PIECES; ++g) w[g] = make_uint2(0, 0);
#pragma unroll
              for (int g = 0; g < PIECES / 4; ++g) sw[g] = 0;
            }
            raw_free();
            if (!wait_all(&empty[st], free_par)) {
              give_up();
              ok = false;
              break;
            }
#pragma unroll
            for (int g = 0; g < PIECES; ++g) {
              const uint32_t sp = e4m3x2_to_f16x2(
                  (uint16_t)(sw[g >> 2] >> (16 * ((g >> 1) & 1))));
              const uint32_t s2 = prmt(sp, 0, (g & 1) ? 0x3232 : 0x1010);
              uint32_t y[8], z[4];
              e2m1x8_to_f16(w[g].x, z);
#pragma unroll
              for (int j = 0; j < 4; ++j) y[j] = mul_f16x2(z[j], s2);
              e2m1x8_to_f16(w[g].y, z);
#pragma unroll
              for (int j = 0; j < 4; ++j) y[4 + j] = mul_f16x2(z[j], s2);
              put(g, y);
            }
          } else {
            // rows are a power of two apart: each reads its pieces in an
            // order of its own, so that eight rows meet all the banks
            const int turn = D == 128 ? r & 7 : (r >> 1) & 3;
            uint4 w[PIECES];
#pragma unroll
            for (int g = 0; g < PIECES; ++g) {
              w[g] = *reinterpret_cast<const uint4 *>(src + 16 * (g ^ turn));
              if (dead) w[g] = make_uint4(0, 0, 0, 0);
            }
            raw_free();
            if (!wait_all(&empty[st], free_par)) {
              give_up();
              ok = false;
              break;
            }
#pragma unroll
            for (int g = 0; g < PIECES; ++g) {
              const uint32_t cw[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
              uint32_t y[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                y[2 * j] = e4m3x2_to_f16x2((uint16_t)cw[j]);
                y[2 * j + 1] = e4m3x2_to_f16x2((uint16_t)(cw[j] >> 16));
              }
              put(g ^ turn, y);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
          if ((rs += 2) >= NR) rs -= NR, rph ^= 1;
        }
      } while (next(sg));
    }
  } else if (!WIDEN && warp < C::SOFT + 4) {
    // ======================= queries ======================================
    int use = 0;
    bool ok = true;
    Seg sg;
    do {
      sg = here();
      for (int t = 0; t < sg.tiles(); ++t, ++use) {
        if (ok && !wait_all(&qempty[q_slot(use)], q_par(use) ^ 1)) {
          give_up();
          ok = false;
        }
        if (ok) load_queries(sg, t, use, tid & 127, 0);
      }
    } while (next(sg));
  } else {
    if constexpr (WIDEN) reg_dec<72>();
    const int bs = p.block_size;
    auto block_of = [&](int b, int lb) {
      int pb = p.block_table[(long)b * p.max_blocks + lb];
      if (pb < 0 || pb >= p.num_blocks) {
        report(p.err, DEVERR_BLOCK);
        pb = 0;  // read a valid block; the result is flagged as wrong
      }
      return pb;
    };
    if (warp == C::kLoad || warp == C::kLoadV) {
      // ===================== copies of K, of V ============================
      // (A warp's copies follow one another at 827 cycles for a swizzled tile
      // of 16 KB, 540 unswizzled, from L2 too; those of two warps overlap.)
      // Pieces of a chunk: boxes of tp.box rows (bf16), or what it has of a
      // block. Chunks are looked up 32 / L at a time: lane l takes piece l % L
      // of chunk l / L of the batch (L: pieces a chunk may have, a power of
      // two), and later issues that piece's copies. L = 32 and more pieces: a
      // lane looks further ones up when it issues.
      int L = 1;
      if constexpr (!WIDEN) {
        L = min(32, kN >> (__ffs(tp.box) - 1));
      } else {
        while (L < 32 && L < (bs % kN == 0   ? 1
                              : kN % bs == 0 ? kN / bs
                                             : kN / bs + 2))
          L <<= 1;
      }
      const int shift = __ffs(L) - 1, lq = lane & (L - 1), batch = 32 >> shift;
      const int mine = lane >> shift, bshift = WIDEN ? 0 : __ffs(tp.box) - 1;
      bool go = true;
      const int q = warp == C::kLoadV;
      int gc = 0;  // chunks so far
      // Rows of a V tile that no pair attends to are zeros, so that 0 times
      // them stays 0. Beside raw rows lie the bits of those attended to, for
      // the warps that widen them. bf16: the copies left such rows as they were,
      // or brought in what lies beside the sequence, or nodes that no mask has. A
      // tile that may have them arrives on a barrier of its own (`land`); rows
      // whose bits are not in `seen` are filled behind the copies of the next
      // one, and before any wait.
      int ends_slot = -1;
      uint32_t seen = 0;  // lane w: of rows [32 w, 32 w + 32)
      uint32_t par = 0;  // parities of `land`, a bit a slot
      auto fill_ends = [&]() {
        if (ends_slot < 0) return;
        const int s = ends_slot;
        ends_slot = -1;
        if (!wait_all(&land[s], par >> s & 1)) {
          go = false;
          return;
        }
        par ^= 1u << s;
        uint8_t *tile = smem + C::KV_OFF + s * C::TILE;
        // a lane a 16-byte piece of a row, AT rows at a time (a loop over the
        // set bits instead: one tree 23.6 us against 20.7, a unit's last tile
        // waits for these stores)
        constexpr int PC = D / 8, AT = 32 / PC;
        const int r0 = lane / PC, e = lane % PC;
        uint8_t *piece = tile + (e >> 3) * C::COLS + r0 * 128 + (e & 7) * 16;
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
          const uint32_t m = ~__shfl_sync(0xffffffffu, seen, w);
          if (m == 0) continue;
          uint8_t *at = piece + (w >> 1) * C::HALF + (w & 1) * 32 * 128;
#pragma unroll
          for (int k = 0; k < 32; k += AT)
            if (m >> r0 >> k & 1)
              *reinterpret_cast<uint4 *>(at + k * 128) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      };
      Seg sg;
      do {
        sg = here();
        const int first =
            q == 1 ? first_seen(p, sg.q, wk.b, lane) : sg.q.lo;
        const int c0 = sg.c0(), c1 = c0 + sg.nch;
        for (int cb = c0; go && cb < c1; cb += batch) {
          // this lane's piece: positions [x0, x1), at row `at` of the cache
          const int c = cb + mine;
          int t0 = 0, t1 = 0;
          auto piece = [&](int i, int &x0, int &x1) -> long {
            if constexpr (!WIDEN) {
              x0 = c * kN + i * tp.box;
              x1 = x0 + tp.box;
              if (i * tp.box >= kN || x1 <= t0 || x0 >= t1) {
                x1 = x0;
                return 0;
              }
            } else {
              // (64 bits: a block that holds position 2^31 - 257 may end past
              // 2^31)
              const long b0 = (long)(t0 / bs + i) * bs;
              x0 = (int)min(max((long)t0, b0), (long)t1);
              x1 = (int)min((long)t1, b0 + bs);
              if (x0 >= x1) {
                x1 = x0;
                return 0;
              }
            }
            const int lb = x0 / bs;
            return ((long)block_of(wk.b, lb) * p.n_kv + sg.h) * bs +
                   (x0 - lb * bs);
          };
          int x0 = 0, x1 = 0;
          long at = 0;
          if (c < c1) {
            t0 = max(c * kN, sg.q.lo);
            t1 = min((c + 1) * kN, sg.q.T);
            if constexpr (DT == DT_MXFP4) {
              // (rows of 72 bytes are copied in pairs; block sizes are even)
              t0 &= ~1;
              t1 = (t1 + 1) & ~1;
            }
            at = piece(lq, x0, x1);
          }
          const int cnt = min(batch, c1 - cb);
          for (int j = 0; go && j < cnt; ++j, ++gc) {
            const int p0 = (cb + j) * kN;
            const int s = WIDEN ? (2 * gc + q) % NR
                          : q   ? C::v_slot(gc)
                                : C::k_slot(gc);
            uint64_t *free = WIDEN ? &rawempty[s] : &empty[s];
            const uint32_t free_par = (WIDEN ? (2 * gc + q) / NR & 1
                                       : q   ? C::v_par(gc)
                                             : C::k_par(gc)) ^
                                      1;
            const bool ends =
                q == 1 && (p0 < first || p0 > sg.q.ctx - kN);
            if constexpr (!WIDEN) {
              if (!__all_sync(0xffffffffu, mbar_test_wait(free, free_par)))
                fill_ends();
            }
            go = go && wait_all(free, free_par);
            if (!go) break;
            if (mine == j) {
              if constexpr (!WIDEN) {
                uint64_t *bar = ends ? &land[s] : &full[s];
                const int n =
                    ((t1 + tp.box - 1) >> bshift) - (t0 >> bshift);
                if (lq == 0)
                  mbar_arrive_expect_tx(bar,
                                        (uint32_t)(n << bshift) * D * 2);
                uint8_t *tile = smem + C::KV_OFF + s * C::TILE;
                const int kv = tp.which[q];
                const CUtensorMap *map = &tp.map[q && tp.far];
                for (int i = lq; i * tp.box < kN; i += L) {
                  int a0 = x0, a1 = x1;
                  long row = at;
                  if (i > lq) row = piece(i, a0, a1);
                  if (a0 >= a1) continue;
                  const int o = i * tp.box;  // row of the chunk
                  uint8_t *dst = tile + (o >> 6) * C::HALF + (o & 63) * 128;
                  if (tp.box == 64) {
                    tma_load_4d(dst, map, 0, (int)row, 0, kv, bar);
                  } else {
#pragma unroll
                    for (int z = 0; z < D / 64; ++z)
                      tma_load_4d(dst + z * C::COLS, map, 0, (int)row, z, kv,
                                  bar);
                  }
                }
              } else {
                constexpr int ROW = row_bytes(D, DT);
                uint8_t *dst = smem + C::RAW_OFF + s * C::RAW;
                const uint8_t *src = q ? p.v : p.k;
                for (int i = lq;; i += L) {
                  int a0 = x0, a1 = x1;
                  long row = at;
                  if (i > lq) row = piece(i, a0, a1);
                  if (a0 < a1)
                    bulk_g2s(dst + (a0 - c * kN) * ROW, src + row * ROW,
                             (uint32_t)(a1 - a0) * ROW, &rawfull[s]);
                  if (L < 32 || (long)(t0 / bs + i + L) * bs >= t1) break;
                }
              }
            }
            __syncwarp();
            auto look = [&]() {
              uint32_t bits = 0;
#pragma unroll 1
              for (int w = 0; w < 4; ++w) {
                const uint32_t x =
                    seen_by_some(p, sg.q, first, p0 + 32 * w, lane);
                if (lane == w) bits = x;
              }
              return bits;
            };
            if constexpr (!WIDEN) {
              fill_ends();
              if (ends) ends_slot = s, seen = look();
            } else {
              if (q == 1) {
                const uint32_t bits = ends ? look() : 0xffffffffu;
                if (lane < 4) seen_v[4 * s + lane] = bits;
                __syncwarp();
              }
              // (copies may have landed by now: the phase ends with this
              // arrival at the earliest, which publishes the bits too)
              if (mine == j && lq == 0)
                mbar_arrive_expect_tx(
                    &rawfull[s], (uint32_t)(t1 - t0) * row_bytes(D, DT));
            }
          }
        }
      } while (next(sg));
      fill_ends();
      if (!go) {
        give_up();
        // every copy that was issued has landed before this CTA gives its
        // shared memory back
        for (int g = max(gc - NS, 0); g < gc; ++g) {
          if constexpr (WIDEN) {
            if (g < gc - NR / 2) continue;
            mbar_wait(&rawfull[(2 * g + q) % NR], (2 * g + q) / NR & 1);
          } else if (g >= gc - (q ? C::VS : C::KS)) {
            const int s = q ? C::v_slot(g) : C::k_slot(g);
            mbar_wait(s == ends_slot ? &land[s] : &full[s],
                      s == ends_slot ? par >> s & 1
                      : q            ? C::v_par(g)
                                     : C::k_par(g));
          }
        }
      }
    } else if (warp == C::kMma || warp == C::kMma + 1) {
      // ===================== MMA issue ====================================
      constexpr uint32_t idS = WIDEN ? umma_idesc_f16(kM, kS, false)
                                     : umma_idesc_bf16(kM, kS, false);
      constexpr uint32_t idO = WIDEN ? umma_idesc_f16(kM, D, true)
                                     : umma_idesc_bf16(kM, D, true);
      const uint32_t q0 = smem_u32(smem + C::Q_OFF);
      const uint32_t kv0 = smem_u32(smem + C::KV_OFF);
      // A step's barriers: V's, complete by then as a rule, is polled; then P's
      // (or Q's), by a suspending wait, which leaves the issue slots to the
      // softmax warps.
      auto poll = [&](uint64_t *bar, uint32_t par) {
        for (int i = 0; i < (1 << 24); ++i)
          if (__all_sync(0xffffffffu, mbar_test_wait(bar, par))) return true;
        return false;
      };
      // One warp a tile; each touches its own tensor memory only. Both see every
      // K tile arrive and every V tile, in their order (a barrier's phases must
      // not pass unseen), and both let go of it: after the products that read it,
      // or at once where the other tile's do.
      const int t = warp - C::kMma;
      int use = 0, gc = 0, gv = 0, seen_k = 0, seen_v = 0;
      bool ok = true;
      Seg sg;
      do {
        sg = here();
        const int nv = uniform(sg.steps(t)), nch = uniform(sg.nch);
        const bool two = uniform(sg.two);
        const int qu = use + (two ? t : 0);
        const uint32_t qa = q0 + q_slot(qu) * C::TILE;
        auto chunk = [&](int v) { return gc + chunk_of(two, t, v); };
        // wait for the tiles up to chunk g
        auto see = [&](int g, int st, uint32_t par) {
          if (!poll(&full[st], par)) return false;
          if (!two && ((g - gc) & 1) != t) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
          }
          return true;
        };
        auto need_k = [&](int g) {
          for (; seen_k <= g; ++seen_k)
            if (!see(seen_k, C::k_slot(seen_k), C::k_par(seen_k))) return false;
          return true;
        };
        auto need_v = [&](int g) {
          for (; seen_v <= g; ++seen_v)
            if (!see(seen_v, C::v_slot(seen_v), C::v_par(seen_v))) return false;
          return true;
        };
        // scores of step v, whose K tile is there
        auto issue_s = [&](int v) {
          const int st = C::k_slot(chunk(v)), buf = v & 1;
          const uint64_t a = umma_desc_sw128(qa, 16, 1024);
          const uint64_t bk =
              umma_desc_sw128(kv0 + st * C::TILE + buf * C::HALF, 16, 1024);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t step = (ks & 3) * 32;
            umma_ss_elect(tbase + kColS + 128 * t + kS * buf,
                          a + (((ks >> 2) * 2 * C::COLS + step) >> 4),
                          bk + (((ks >> 2) * C::COLS + step) >> 4), idS,
                          ks > 0 ? 1u : 0u);
          }
          umma_commit_elect(&sfull[2 * t + buf]);
          if (buf == 1) umma_commit_elect(&empty[st]);  // the chunk's last step
        };
        // both tiles' query slots are seen and let go of by both warps
        for (int i = 0; ok && i <= (int)two; ++i)
          ok = wait_all(&qfull[q_slot(use + i)], q_par(use + i));
        // two steps of scores ahead; then per step the product with V and the
        // scores of the step after next, into the buffer P just left
        if (ok && nv > 0) {
          ok = need_k(chunk(0));
          tc_fence_after();
          if (ok) {
            issue_s(0);
            issue_s(1);
          }
        }
        for (int v = 0; ok && v < nv; ++v) {
          const int buf = v & 1, st = C::v_slot(chunk(v));
          if (v == nv - 2) {
            // the unit's scores are all issued: its queries are free
            for (int i = 0; i <= (int)two; ++i)
              umma_commit_elect(&qempty[q_slot(use + i)]);
          }
          ok = need_v(chunk(v)) &&
               wait_all(&pfull[2 * t + buf], ((gv + v) >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bv = umma_desc_sw128(
              kv0 + st * C::TILE + buf * C::HALF, C::COLS, 1024);
#pragma unroll
          for (int kk = 0; kk < kS / 16; ++kk)
            umma_ts_elect(tbase + kColO + D * t,
                          tbase + kColS + 128 * t + kS * buf + kk * 8,
                          bv + (uint64_t)((kk * 2048) >> 4), idO,
                          (v > 0 || kk > 0) ? 1u : 0u);
          umma_commit_elect(&pvdone[t]);
          if (buf == 1) umma_commit_elect(&empty[st]);
          if (v == nv - 1) umma_commit_elect(&odone[t]);
          if (v + 2 < nv) {
            ok = need_k(chunk(v + 2));
            tc_fence_after();
            if (ok) issue_s(v + 2);
          }
        }
        if (ok && nv == 0)
          for (int i = 0; i <= (int)two; ++i)
            umma_commit_elect(&qempty[q_slot(use + i)]);
        // the other tile's last ones too
        ok = ok && need_k(gc + nch - 1) && need_v(gc + nch - 1);
        use += two ? 2 : 1;
        gc += nch;
        gv += nv;
      } while (ok && next(sg));
      if (!ok) give_up();
      // every MMA issued has completed before the dealloc
      umma_commit_elect(drain);
      mbar_wait(drain, 0);
    }
  }
  tc_fence_before();
  __syncthreads();  // every read of tensor memory is done
  if (warp == C::kMma) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int DT, int D, int QS>
cudaError_t launch_attend_t(const TcParams &tp, cudaStream_t s) {
  using C = ACfg<DT, D, QS>;
  static bool done[64] = {};
  auto kern = attend_tc_kernel<DT, D, QS>;
  const cudaError_t e = set_smem_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(tp.p.n_splits), dim3(C::THREADS), C::SMEM, s, 1,
                    tp);
}

}  // namespace

// Caches whose rows are widened (attend_widen.cu); `one`: no unit of the
// launch has two tiles.
cudaError_t launch_attend_widen(const TcParams &tp, bool one, cudaStream_t s);

}  // namespace kvd
