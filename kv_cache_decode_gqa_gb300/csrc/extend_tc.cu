// Attention of several new rows a sequence over an MXFP4 cache on the
// 5th-generation tensor cores (kvd_gqa_extend with more than 16 (row, query
// head) pairs a kv head: prompts, chunks of prompts, drafts of wide groups).
//
// The (row, head) pairs of a kv head are numbered row-major, pair f = row *
// G + head, so any group size G fills the MMA's M. A CTA takes a block of up
// to 256 pairs -- two M = 128 tiles -- against chunks of 128 positions:
//   S = Q K^T   (A = Q in shared memory, B = K chunk, K-major)
//   O += P V    (A = P in tensor memory, over S; B = V chunk, MN-major)
// with S, P and O of each tile in 128 + 128 columns of tensor memory (512 in
// all) and one softmax thread per pair (tensor-memory lane). A tile's S lies
// in two buffers of 64 positions: while the softmax turns one into P, the
// tensor core does PV of the other and the scores that follow it, for this
// tile and for the other one. A block of at most 128 pairs has one tile only;
// then both halves work for it, on even and odd chunks, and their states are
// merged at the end. Where a sequence may have more than 256 pairs a kv head,
// two CTAs take blocks of 512 (cta_group::2, M = 256): each widens half of
// every chunk's K rows and half of V's columns, and the products read both
// halves.
//
// What bounds it: prompts do 4 * 128 multiply-adds' flops a (pair, position)
// at the f16 rate (512 cycles an M = N = K = 128 product); a few rows over a
// long cache read 144 bytes a position. Either way 256 codes of a position
// are widened once per block, by eight warps: a row a thread, 8 codes at a
// time, times the group's E4M3 scale (exact in f16), into the 128-byte-
// swizzled tiles that both products read. Raw rows come through a ring of
// bulk copies, so that the widening never waits for HBM.
//
// Measured: 1,021 rows over 32,000 positions, 56 heads of 8 kv heads, in 705
// us (1,350 TFLOP/s, 70% of cuBLAS's bf16 rate); whole prompts of 7,001 rows
// in two sequences, 64 heads, in 430 us; 4 rows of each of 16 sequences over
// 8,700 positions (160 MB) in 102 us (32 pairs: 32 of a tile's 128 lanes, so
// that one softmax warp of each group does all of its exponentials and three
// quarters of the products are padding). In a less even split (797 us) the
// first took 627 us without the exponentials, 779 without the widening, 744
// without most of the products, 478 with none of them: it is the time from a
// product's end to the softmax and from P back to the next product that is
// left, one after the other in each of a tile's two buffers. (Softmax groups
// that take turns on named barriers: 850 us; one S buffer of 128 positions a
// tile: the same; K and V handed over by halves of a chunk: the second took
// 6% longer; a third K tile in the place of an unused second tile: 4% slower
// for the few rows, for the ring of raw rows shrinks.)
//
// The softmax keeps a reference per pair, 2^7 below a maximum, and moves it
// only when a chunk exceeds that maximum by more than 2^8 (the accumulator is
// rescaled then, in tensor memory): P stays below 2^15 and its largest is at
// least 2^7, so that f16 drops only what is 2^-32 of it and below (see
// extend_few.cu), and the final division by the sum (fp32, of the same
// exponentials) takes the reference out again. Queries are scaled by a power
// of two per (row, head) into f16 (see extend_few.cu).
//
// Warp roles (640 threads, one CTA per SM; registers are moved from the
// launch's 96 a thread, 61,440, to 128 for the softmax and 72 for the others,
// 60,416):
//   warps 0-3, 4-7     softmax of tile 0 and 1, query load, epilogue
//   warps 8-11, 12-15  widening of K and of V (one group for both took 3,300
//                      cycles a chunk, the softmax and products 2,300)
//   warp 16            bulk copies of cached rows
//   warps 17, 18       MMA issue of tile 0 and 1 (17: tensor memory)
#include <algorithm>
#include <climits>
#include <cmath>

#include "prompt_common.cuh"
#include "tcgen05_pair.cuh"

namespace kvd {
namespace {

constexpr int kD = 128;
constexpr int kRow = 72;             // bytes of a cached row
constexpr int kM = 128;              // pairs per tile
constexpr int kN = kExtendChunk;     // positions per chunk
constexpr int kS = kN / 2;           // positions per product (half a chunk)
constexpr int kTile = 128 * 256;     // a 128 x 128 f16 operand tile, 32 KB
constexpr int kHalf = 128 * 128;     // its 64-column half
constexpr int kRaw = kN * kRow;      // raw K (or V) rows of a chunk
constexpr int kThreads = 640;
constexpr int kWiden0 = 8, kLoadWarp = 16, kMmaWarp = 17;
constexpr int kSoftBar = 1;
constexpr float kHead = 7.f;         // log2 units it lies below the maximum
constexpr float kSlack = 8.f;        // and may lag by

// CTAS = 1 or 2 CTAs share a block's chunks (2: a cta_group::2 pair).
// Shared memory: Q tiles, K ring, V ring (2 each), raw ring.
template <int CTAS>
struct TCfg {
  static constexpr int ROWS = CTAS * kExtendRows;  // pairs per block
  static constexpr int KV = kTile / CTAS;    // this CTA's part of a K, V tile
  // 64-column half of its K part
  static constexpr int KHALF = kHalf / CTAS;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * kTile;
  static constexpr int V_OFF = K_OFF + 2 * KV;
  static constexpr int RAW_OFF = V_OFF + 2 * KV;
  // raw slots: one CTA has three, and three more in Q tile 1 when it is
  // unused
  static constexpr int OWN_SLOTS = CTAS == 1 ? 3 : 6;
  static constexpr int SLOTS = 6;
  static constexpr int F_OFF = RAW_OFF + OWN_SLOTS * kRaw;  // float [4][128]
  static constexpr int BAR_OFF = F_OFF + 4 * kM * 4;
  static constexpr int BARS = 2 * SLOTS + 8 + 10 + 2;
  static constexpr int FLAG_OFF = BAR_OFF + BARS * 8;  // int [8]
  static constexpr int SCAN_OFF = FLAG_OFF + 32;       // int [20]
  static constexpr int SMEM = SCAN_OFF + 128;
  static_assert(3 * kRaw <= kTile && SMEM <= 227 * 1024, "shared memory");
};

// Tensor memory: two score buffers of 64 columns a tile, then the outputs.
constexpr uint32_t kColS = 0, kColO = 256;         // + 128 * tile

// 16-byte piece c (0..7) of row r in a 128-byte-swizzled 64-column half.
__device__ __forceinline__ uint32_t sw128(int r, int c) {
  return (uint32_t)((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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

// What a sequence's blocks are computed from.
struct Seq {
  int n, T;  // its rows and visible length
  int s;     // its first visible position
};

__device__ __forceinline__ Seq seq_at(const ExtendParams &p, int b) {
  Seq q;
  q.n = seq_rows(p, b);
  q.T = min(max(p.seq_lens[b], 0), p.max_seq_len);
  q.s = p.win_start ? max(p.win_start[b], 0) : 0;
  return q;
}

// A row block: the pairs [f0, f1) of block `mb` of a sequence, and the
// positions [lo, hi) they see.
struct Block {
  int f0, f1;
  int lo, hi;
};

__device__ __forceinline__ Block block_at(const ExtendParams &p, const Seq &q,
                                          int mb, int G) {
  Block k;
  k.f0 = mb * p.block_rows;
  k.f1 = min(k.f0 + p.block_rows, q.n * G);
  const int first = q.T - q.n + k.f0 / G, last = q.T - q.n + (k.f1 - 1) / G;
  k.lo = p.window > 0 ? max(q.s, window_lo(p, first)) : q.s;
  k.hi = max(last + 1, 0);
  return k;
}

// Chunks [c0, c1) that a block's positions lie in.
__device__ __forceinline__ void block_chunks(const Block &k, int &c0,
                                             int &c1) {
  c0 = k.lo / kN;
  c1 = k.lo < k.hi ? (k.hi + kN - 1) / kN : c0;
}

// Equal parts, of at most `per` chunks (0: one part), of a block's n chunks.
__device__ __forceinline__ int block_parts(int per, int n) {
  return per > 0 ? max((n + per - 1) / per, 1) : 1;
}

template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1)
    extend_tc_kernel(const __grid_constant__ ExtendParams p) {
  using C = TCfg<CTAS>;
  constexpr bool PAIR = CTAS == 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  float *fs = reinterpret_cast<float *>(smem + C::F_OFF);
  uint64_t *rawfull = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
  uint64_t *rawempty = rawfull + C::SLOTS;
  uint64_t *kfull = rawempty + C::SLOTS;  // [2] each
  uint64_t *kempty = kfull + 2;
  uint64_t *vfull = kempty + 2;
  uint64_t *vempty = vfull + 2;
  uint64_t *sfull = vempty + 2;  // [tile][buffer]
  uint64_t *pfull = sfull + 4;   // [tile][buffer]
  uint64_t *pvdone = pfull + 4;  // [tile]
  uint64_t *qfull = pvdone + 2;
  uint64_t *odone = qfull + 1;
  // [0] tensor memory's address, [1] first_descent, [2 ..] s_blk
  int *flags = reinterpret_cast<int *>(smem + C::FLAG_OFF);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(flags);
  // this CTA's sequence, its block of it, and the sequence's Seq
  int *s_blk = flags + 2;
  int *s_scan = reinterpret_cast<int *>(smem + C::SCAN_OFF);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.n_h / p.n_kv;

  pdl_wait();
  pdl_trigger();  // after the wait: the merge launch never overlaps this
                  // launch's predecessor
  // ---- which block: a scan of the sequences' block counts --------------
  // The last blocks come first: under the causal mask they are the longest.
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int item = (int)blockIdx.x / CTAS;  // the same for a pair's CTAs
  const int h = item % p.n_kv;
  const int want = item / p.n_kv;
  if (tid == 0) s_blk[0] = -1;
  {
    int cnt[2], sum, x, end = p.batch;
    Seq sq[2];
    while (true) {
      bool broken = false;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = 2 * tid + j;
        sq[j] = Seq{0, 0, 0};
        if (b < p.batch) {
          sq[j] = seq_at(p, b);
          broken |= b < end && descends(p, b);
        }
        if (b >= end) sq[j].n = 0;
      }
      sum = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int b = 2 * tid + j;
        cnt[j] = (int)(((long)sq[j].n * G + C::ROWS - 1) / C::ROWS);
        if (b < p.batch && blockIdx.x == 0 && blockIdx.y == 0) {
          if (sq[j].n == 0 && p.row_start &&
              p.row_start[b] != p.row_start[b + 1])
            report(p.err, DEVERR_LEN);
          if (p.seq_lens[b] > p.max_seq_len) report(p.err, DEVERR_LEN);
        }
        sum += cnt[j];
      }
      x = sum;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (lane == 31) s_scan[warp] = x;
      if (!__syncthreads_or(broken)) break;
      end = first_descent(p, flags + 1);
    }
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    int excl = before + x - sum;
    const int mine = total - 1 - want;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (mine >= excl && mine < excl + cnt[j]) {
        s_blk[0] = 2 * tid + j;
        s_blk[1] = mine - excl;
        s_blk[2] = sq[j].n;
        s_blk[3] = sq[j].T;
        s_blk[4] = sq[j].s;
      }
      excl += cnt[j];
    }
  }
  __syncthreads();
  const int b = s_blk[0], mb = s_blk[1];
  if (b < 0) return;  // past the batch's blocks
  const Seq q = {s_blk[2], s_blk[3], s_blk[4]};
  const Block k = block_at(p, q, mb, G);
  int c0, c1;
  block_chunks(k, c0, c1);
  const int parts = block_parts(p.chunks_per_split, c1 - c0);
  const int per = (c1 - c0 + parts - 1) / parts;
  const int part = blockIdx.y;
  if (part >= parts) return;
  c0 += part * per;
  c1 = min(c1, c0 + per);
  const int nch = c1 - c0;
  const int np = k.f1 - k.f0;  // pairs
  const long row0 = p.row_start ? p.row_start[b] : b;
  // output row of pair f: query row f / G, head h G + f % G
  auto out_row = [&](int f) {
    return (row0 + f / G) * p.n_h + (long)h * G + f % G;
  };
  if (nch <= 0) {  // nothing is seen (parts is 1)
    for (int i = rank * kThreads + tid; i < np * (kD / 8);
         i += CTAS * kThreads)
      reinterpret_cast<uint4 *>(p.out + out_row(k.f0 + i / (kD / 8)) *
                                            kD)[i % (kD / 8)] =
          make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = rank * kThreads + tid; i < np; i += CTAS * kThreads)
        p.lse[out_row(k.f0 + i)] = -INFINITY;
    return;
  }
  // the swizzled tiles assume 1 KB atoms (every CTA sees the same layout)
  if ((smem_u32(smem) & 1023u) != 0) {
    if (tid == 0) report(p.err, DEVERR_TIMEOUT);
    return;
  }
  const bool two = PAIR || np > kM;
  const int nraw = two ? C::OWN_SLOTS : C::SLOTS;
  // Step v of tile t: half v & 1 of a chunk -- chunk v / 2 of the range for
  // two tiles, chunks t, t + 2, ... for one tile's two halves
  auto chunk_of = [&](int t, int v) { return two ? v >> 1 : (v & ~1) + t; };
  auto steps_of = [&](int t) { return two ? 2 * nch : (nch - t + 1) & ~1; };

  if (tid == 0) {
    for (int i = 0; i < C::SLOTS; ++i) {
      mbar_init(&rawfull[i], 1);
      mbar_init(&rawempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], 4 * CTAS);
      mbar_init(&kempty[i], two ? 2 : 1);  // one commit a tile
      mbar_init(&vfull[i], 4 * CTAS);
      mbar_init(&vempty[i], two ? 2 : 1);
      mbar_init(&pvdone[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4 * CTAS);
    }
    mbar_init(qfull, CTAS * (two ? 8 : 4));
    mbar_init(odone, 2);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    if constexpr (PAIR) {
      tmem2_alloc(s_tmem, 512);
      tmem2_relinquish();
    } else {
      tmem_alloc(s_tmem, 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // the other CTA's barriers too
  tc_fence_after();
  const uint32_t tbase = *s_tmem;
  auto raw_slot = [&](int s) {
    return smem + (s < C::OWN_SLOTS
                       ? C::RAW_OFF + s * kRaw
                       : C::Q_OFF + kTile + (s - C::OWN_SLOTS) * kRaw);
  };
  // Every wait is bounded; a role that gives up leaves its loop, and the
  // others follow when their own waits run out. (A flag to leave earlier
  // would cost every wait a shared-memory load: 200 to 300 cycles here.)
  auto give_up = [&]() {
    if (lane == 0) report(p.err, DEVERR_TIMEOUT);
  };
  auto wait_all = [&](uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
  };
  // Arrivals that the MMA warps (CTA 0's in a pair) wait for, and commits that
  // the roles of every CTA wait for. CTA 1's tiles in shared memory (Q, K, V)
  // are released at cluster scope, ahead of their use: 434 to 440 us for the
  // prompts (in a graph), 697 to 699 for the chunk. P, on the way from one
  // product to the next, lies in tensor memory and needs the threads' order
  // only (released at cluster scope as well: 537 and 970 us; relayed by CTA
  // 1's own MMA warps: 477 and 842; without pairs: 475 and 792; released in
  // CTA 0, which needs none either: 451 and 726).
  auto arrive_mma = [&](uint64_t *bar) {
    if (PAIR && rank != 0)
      mbar_arrive_remote(cluster_saddr(bar, 0));
    else
      mbar_arrive(bar);
  };
  auto arrive_p = [&](uint64_t *bar) {
    if constexpr (PAIR)
      mbar_arrive_remote_relaxed(cluster_saddr(bar, 0));
    else
      mbar_arrive(bar);
  };
  auto commit = [&](uint64_t *bar) {
    if constexpr (PAIR)
      umma2_commit_elect(bar);
    else
      umma_commit_elect(bar);
  };

  if (warp < kWiden0) {
    // ======================= softmax ======================================
    reg_inc<128>();
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // pair of the tile
    // pair of the block (a pair of CTAs: tile t's first half is CTA 0's)
    const int ri = two ? (t * CTAS + rank) * kM + r : r;
    const bool live = ri < np;
    const int f = k.f0 + ri;
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    // positions this pair sees (a pair that does not exist: all, so that its
    // warp masks nothing for it; its query is 0 and nothing of it is stored)
    int vlo = 0, vhi = INT_MAX;
    if (live) {
      const int pos = q.T - q.n + f / G;
      vhi = max(pos + 1, 0);
      vlo = q.s;
      if (p.window > 0) vlo = max(vlo, window_lo(p, pos));
    }
    // ---- the pair's query, scaled into f16 (tile t, or both halves' one)
    float sl;
    {
      uint4 x[16];
      uint32_t m = 0;
      const uint16_t *src = p.q + (row0 + f / G) * p.q_rs +
                            ((long)h * G + f % G) * p.q_hs;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        x[c] = live ? reinterpret_cast<const uint4 *>(src)[c]
                    : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        m = __vmaxu2(m, __vmaxu2(x[c].x & 0x7fff7fffu, x[c].y & 0x7fff7fffu));
        m = __vmaxu2(m, __vmaxu2(x[c].z & 0x7fff7fffu, x[c].w & 0x7fff7fffu));
      }
      m = max(m & 0xffffu, m >> 16);
      const int e = row_exponent(m);
      const float sc = __uint_as_float((uint32_t)e << 23);
      sl = fmaxf(p.scale_log2 * exp2f((float)(127 - e)), 1.17549435e-38f);
      if (two || t == 0) {
        uint8_t *qt = smem + C::Q_OFF + (two ? t * kTile : 0);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint4 w;
          w.x = pack_f16x2(bf16lo(x[c].x) * sc, bf16hi(x[c].x) * sc);
          w.y = pack_f16x2(bf16lo(x[c].y) * sc, bf16hi(x[c].y) * sc);
          w.z = pack_f16x2(bf16lo(x[c].z) * sc, bf16hi(x[c].z) * sc);
          w.w = pack_f16x2(bf16lo(x[c].w) * sc, bf16hi(x[c].w) * sc);
          *reinterpret_cast<uint4 *>(qt + (c >> 3) * kHalf +
                                     sw128(r, c & 7)) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_mma(qfull);
      }
    }
    const bool warp_live = __any_sync(0xffffffffu, live);
    float ref = -INFINITY, l = 0.f;
    const uint64_t sl2 = pack_f32x2(sl, sl);
    const int nv = steps_of(t);
    for (int v = 0; v < nv; ++v) {
      const int buf = v & 1;
      const int pos0 = (c0 + chunk_of(t, v)) * kN + buf * kS;
      if (!wait_all(&sfull[2 * t + buf], (v >> 1) & 1)) {
        give_up();
        break;
      }
      tc_fence_after();
      if (warp_live) {
        uint32_t x[2][32];
        const uint32_t ts = tl + kColS + 128 * t + kS * buf;
#pragma unroll
        for (int g = 0; g < 2; ++g) tmem_ld32(ts + 32 * g, x[g]);
#pragma unroll
        for (int g = 0; g < 2; ++g) tmem_wait_ld(x[g]);
        // columns [a, z) are seen
        const int a = vlo - pos0, z = vhi - pos0;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // groups of 32 columns that some pair of the warp sees in part
          if (__any_sync(0xffffffffu, a > 32 * g || z < 32 * g + 32)) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * g + i < a || 32 * g + i >= z)
                x[g][i] = 0xff800000u;  // -inf
          }
        }
        float mx[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t *y = &x[g >> 1][16 * (g & 1)];
          mx[g] = fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
#pragma unroll
          for (int i = 2; i < 16; i += 2)
            mx[g] = max3(mx[g], __uint_as_float(y[i]),
                         __uint_as_float(y[i + 1]));
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
            if (!wait_all(&pvdone[t], (v - 1) & 1)) {
              give_up();
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              uint32_t o[16];
              const uint32_t to = tl + kColO + 128 * t + 16 * g;
              tmem_ld16(to, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              tmem_st16(to, o);
            }
          }
        }
        const float mu = ref == -INFINITY ? 0.f : ref;
        const uint64_t mu2 = pack_f32x2(-mu, -mu);
        uint64_t ls[2] = {0, 0};
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0, e1;
            unpack_f32x2(
                fma_f32x2(pack_f32x2(__uint_as_float(x[g][2 * i]),
                                     __uint_as_float(x[g][2 * i + 1])),
                          sl2, mu2),
                e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            ls[i & 1] = add_f32x2(ls[i & 1], pack_f32x2(e0, e1));
            pk[i] = pack_f16x2(e0, e1);
          }
          tmem_st16(ts + 16 * g, pk);
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
      if (lane == 0) arrive_p(&pfull[2 * t + buf]);
    }
    // ---- epilogue --------------------------------------------------------
    const bool ok = wait_all(odone, 0);
    if (!ok) give_up();
    tc_fence_after();
    float w0 = 1.f, w1 = 0.f, M = ref, L = l;
    if (!two) {
      // the halves' states of pair r: this thread's own and the other's
      fs[t * kM + r] = ref;
      fs[(2 + t) * kM + r] = l;
      named_sync(kSoftBar, 2 * kM);
      const float ra = fs[r], rb = fs[kM + r];
      M = fmaxf(ra, rb);
      const float mu = M == -INFINITY ? 0.f : M;
      w0 = ex2(ra - mu);
      w1 = ex2(rb - mu);
      L = fs[2 * kM + r] * w0 + fs[3 * kM + r] * w1;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float lse =
        L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
    const long at = live ? out_row(f) : 0;
    // two tiles: all 128 columns of the tile's pair; one: the halves write
    // 64 columns each
    const int ncol = two ? kD : kD / 2;
    const int col0 = two ? 0 : t * (kD / 2);
    const uint32_t ta = tl + kColO + (two ? 128 * t : 0) + col0;
    const bool second = !two && nch > 1;
    if (warp_live && ok) {
#pragma unroll 1
      for (int g = 0; g < ncol; g += 32) {
        uint32_t o[32];
        tmem_ld32(ta + g, o);
        tmem_wait_ld(o);
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i)
          y[i] = __uint_as_float(o[i]) * (two ? inv : w0 * inv);
        if (second) {
          tmem_ld32(ta + 128 + g, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            y[i] = fmaf(__uint_as_float(o[i]), w1 * inv, y[i]);
        }
        if (live) {
          if (parts == 1) {
            uint4 *dst =
                reinterpret_cast<uint4 *>(p.out + at * kD + col0 + g);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]),
                                  pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                  pack_bf16x2(y[8 * i + 4], y[8 * i + 5]),
                                  pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
          } else {
            float4 *dst = reinterpret_cast<float4 *>(
                p.ws_o + ((long)part * p.rows * p.n_h + at) * kD + col0 + g);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2],
                                   y[4 * i + 3]);
          }
        }
      }
      if (live && (two || t == 0)) {
        if (parts > 1)
          p.ws_lse[(long)part * p.rows * p.n_h + at] = lse;
        else if (p.lse)
          p.lse[at] = lse;
      }
    }
  } else if (warp < kLoadWarp) {
    // ======================= widening =====================================
    reg_dec<72>();
    // A thread widens a row of the chunk, 128 columns; in a pair 64: CTA
    // `rank` has the K rows [32 rank, + 32) of either half of the chunk (N of
    // the scores' products) and V columns [64 rank, + 64) (N of the outputs')
    const int tw = (tid - kWiden0 * 32) & 127;
    const bool is_v = warp >= kWiden0 + 4;
    constexpr int kGroups = 8 / CTAS;  // 16-column groups a thread
    const int r = PAIR && !is_v ? tw & 63 : tw;        // row of the raw unit
    const int g0 = !PAIR ? 0 : is_v ? 4 * rank : 4 * (tw >> 6);
    // its position in the chunk
    const int cpos = PAIR && !is_v ? (r & 31) + 64 * (r >> 5) + 32 * rank : r;
    const uint32_t half = PAIR ? C::KHALF : kHalf;     // of the tile written
    uint64_t *tfull = is_v ? vfull : kfull, *tempty = is_v ? vempty : kempty;
    // K rows are raw units 0, 2, 4, ..., V rows 1, 3, 5, ...
    int rs = is_v, rph = 0;
    for (int i = 0; i < nch; ++i) {
      const int st = i & 1, ph = (i >> 1) & 1;
      if (!wait_all(&rawfull[rs], rph)) {
        give_up();
        break;
      }
      const uint8_t *src = raw_slot(rs) + r * kRow;
      uint2 w[kGroups];
      uint32_t sw[kGroups / 4];  // scales, four a word
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        w[g] = *reinterpret_cast<const uint2 *>(src + 8 * (g0 + g));
#pragma unroll
      for (int g = 0; g < kGroups / 4; ++g)
        sw[g] = *reinterpret_cast<const uint32_t *>(src + 64 + g0 + 4 * g);
      const int pos = (c0 + i) * kN + cpos;
      if (pos < k.lo || pos >= k.hi) {
        // a row that was not copied, or that no pair sees: zeros, so that 0
        // times it stays 0
#pragma unroll
        for (int g = 0; g < kGroups; ++g) w[g] = make_uint2(0, 0);
#pragma unroll
        for (int g = 0; g < kGroups / 4; ++g) sw[g] = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&rawempty[rs]);
      if ((rs += 2) >= nraw) rs -= nraw, rph ^= 1;
      // the tile's last reader is done (a fresh barrier passes parity 1)
      if (!wait_all(&tempty[st], ph ^ 1)) {
        give_up();
        break;
      }
      uint8_t *dst = smem + (is_v ? C::V_OFF : C::K_OFF) + st * C::KV;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const uint32_t sp = e4m3x2_to_f16x2(
            (uint16_t)(sw[g >> 2] >> (16 * ((g >> 1) & 1))));
        const uint32_t s2 = prmt(sp, 0, (g & 1) ? 0x3232 : 0x1010);
        const uint32_t cw[2] = {w[g].x, w[g].y};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t x[4];
          e2m1x8_to_f16(cw[q], x);
          uint4 y;
          y.x = mul_f16x2(x[0], s2);
          y.y = mul_f16x2(x[1], s2);
          y.z = mul_f16x2(x[2], s2);
          y.w = mul_f16x2(x[3], s2);
          // 16-byte piece of the row: of the CTA's own columns for V
          const int c = 2 * ((PAIR && is_v ? 0 : g0) + g) + q;
          *reinterpret_cast<uint4 *>(dst + (c >> 3) * half +
                                     sw128(r, c & 7)) = y;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_mma(&tfull[st]);
    }
  } else {
    reg_dec<72>();
    if (warp == kLoadWarp) {
      // ===================== bulk copies ==================================
      // In alternation K and V of a chunk. Chunks are looked up 32 / L at a
      // time: lane l takes block l % L of chunk l / L of the batch (L: blocks
      // a chunk may touch, a power of two), and later issues that block's
      // copies. Attended positions are widened to even bounds (rows of 72
      // bytes are copied in pairs; block sizes are even). L = 32 and more
      // blocks (of 2 positions): a lane takes further ones when it issues.
      const int bs = p.block_size;
      auto block_of = [&](int lb) {
        int pb = p.block_table[(long)b * p.max_blocks + lb];
        if (pb < 0 || pb >= p.num_blocks) {
          report(p.err, DEVERR_BLOCK);
          pb = 0;  // read a valid block; the result is flagged as wrong
        }
        return pb;
      };
      int L = 1;
      while (L < 32 && L < (bs % kN == 0   ? 1
                            : kN % bs == 0 ? kN / bs
                                           : kN / bs + 2))
        L <<= 1;
      const int lq = lane & (L - 1), batch = 32 / L;
      int s = 0, ph = 1, units = 0;
      bool go = true;
      for (int cb = c0; go && cb < c1; cb += batch) {
        // this lane's block: its positions [x0, x1) of its chunk, and where
        // position 0 would lie in the cache if the block went back that far
        const int c = cb + lane / L;
        int t0 = 0, t1 = 0, x0 = 0, x1 = 0;
        long at = 0;
        if (c < c1) {
          t0 = max(c * kN, k.lo) & ~1;
          t1 = (min((c + 1) * kN, k.hi) + 1) & ~1;
          const int lb = t0 / bs + lq;
          x0 = max(t0, lb * bs);
          x1 = min(t1, (lb + 1) * bs);
          if (x0 < x1)
            at = (((long)block_of(lb) * p.n_kv + h) * bs - (long)lb * bs) *
                 kRow;
        }
        const int cnt = min(batch, c1 - cb);
        for (int j = 0; go && j < cnt; ++j) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // K, V
            go = go && wait_all(&rawempty[s], ph);
            if (!go) break;
            if (lane / L == j) {
              uint8_t *dst = raw_slot(s);
              const uint8_t *src = q ? p.v : p.k;
              // (copies may land before the expectation is set: the phase
              // ends with that arrival at the earliest)
              uint64_t *bar = &rawfull[s];
              // positions [u0, u1), of which this lane's block has some, to
              // rows (position - base) of the raw unit
              auto copy = [&](int u0, int u1, int base) {
                for (int m = lq; ; m += L) {
                  int a0 = max(u0, x0), a1 = min(u1, x1);
                  long off = at;
                  if (m > lq) {  // blocks of 2 positions: a lane has several
                    const int lb = t0 / bs + m;
                    a0 = max(u0, lb * bs), a1 = min(u1, (lb + 1) * bs);
                    if (a0 < a1)
                      off = (((long)block_of(lb) * p.n_kv + h) * bs -
                             (long)lb * bs) * kRow;
                  }
                  if (a0 < a1)
                    bulk_g2s(dst + (a0 - base) * kRow,
                             src + off + (long)a0 * kRow,
                             (uint32_t)(a1 - a0) * kRow, bar);
                  if (L < 32 || (m + L) * bs + t0 / bs * bs >= t1) break;
                }
              };
              if (PAIR && q == 0) {
                // this CTA's 32 positions of either half of the chunk
                const int p0 = c * kN + 32 * rank, p1 = p0 + kS;
                const int a0 = max(t0, p0), a1 = max(min(t1, p0 + 32), a0);
                const int b0 = max(t0, p1), b1 = max(min(t1, p1 + 32), b0);
                if (lq == 0)
                  mbar_arrive_expect_tx(
                      bar, (uint32_t)(a1 - a0 + b1 - b0) * kRow);
                copy(a0, a1, p0);
                copy(b0, b1, p1 - 32);
              } else {
                if (lq == 0)
                  mbar_arrive_expect_tx(bar, (uint32_t)(t1 - t0) * kRow);
                copy(t0, t1, c * kN);
              }
            }
            __syncwarp();
            ++units;
            if (++s == nraw) s = 0, ph ^= 1;
          }
        }
      }
      if (!go) {
        give_up();
        // every copy that was issued has landed before this CTA gives its
        // shared memory back
        for (int i = 0; i < nraw && i < units; ++i) {
          const int u = units - 1 - i;
          mbar_wait(&rawfull[u % nraw], (u / nraw) & 1);
        }
      }
    } else if ((warp == kMmaWarp || warp == kMmaWarp + 1) && rank == 0) {
      // ===================== MMA issue ====================================
      constexpr uint32_t idS = umma_idesc_f16(CTAS * kM, kS, false);
      constexpr uint32_t idO = umma_idesc_f16(CTAS * kM, kD, true);
      const uint32_t q0 = smem_u32(smem + C::Q_OFF);
      const uint32_t k0 = smem_u32(smem + C::K_OFF);
      const uint32_t v0 = smem_u32(smem + C::V_OFF);
      // A step's barriers: first those that are complete by then as a rule,
      // one a lane; last the one that is not (P, or Q), by a suspending wait,
      // which leaves the issue slots to the softmax warps.
      auto wait3 = [&](uint64_t *b0, uint32_t p0, uint64_t *b1, uint32_t p1,
                       uint64_t *b2, uint32_t p2) -> bool {
        if (b1 != nullptr || b2 != nullptr) {
          uint64_t *bar = lane == 1 ? b1 : lane == 2 ? b2 : nullptr;
          const uint32_t par = lane == 1 ? p1 : p2;
          bool done = bar == nullptr;
          int i = 0;
          for (; i < (1 << 24); ++i) {
            done = done || mbar_test_scope<PAIR>(bar, par);
            if (__all_sync(0xffffffffu, done)) break;
          }
          if (i == (1 << 24)) return false;
        }
        return __all_sync(0xffffffffu, mbar_wait_scope<PAIR>(b0, p0));
      };
      // One warp a tile: a wait costs 300 cycles and more here even when its
      // phase is over (the shared memory pipe is busy with the tiles), and
      // the tiles' waits then overlap. Each tile touches its own tensor
      // memory only; a K or V tile is free when both have read it.
      const int t = warp - kMmaWarp;
      const int nv = steps_of(t);
      // scores of step v, whose K tile is there
      auto issue_s = [&](int v) {
        const int st = chunk_of(t, v) & 1, buf = v & 1;
        const uint64_t a = umma_desc_sw128(q0 + (two ? t * kTile : 0), 16,
                                           1024);
        // rows of this half of the chunk: 64, or 32 in each CTA of a pair
        const uint64_t bk = umma_desc_sw128(
            k0 + st * C::KV + buf * (kS / CTAS) * 128, 16, 1024);
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
          const uint32_t step = (ks & 3) * 32;
          const uint64_t ao = a + (((ks >> 2) * kHalf + step) >> 4);
          const uint64_t bo = bk + (((ks >> 2) * C::KHALF + step) >> 4);
          const uint32_t d = tbase + kColS + 128 * t + kS * buf;
          if constexpr (PAIR)
            umma2_ss_elect(d, ao, bo, idS, ks > 0 ? 1u : 0u);
          else
            umma_ss_elect(d, ao, bo, idS, ks > 0 ? 1u : 0u);
        }
        commit(&sfull[2 * t + buf]);
        if (buf == 1) commit(&kempty[st]);  // the chunk's last step
      };
      // the K barrier that step v waits for (a chunk's first step only)
      auto kbar = [&](int v) -> uint64_t * {
        return v < nv && (v & 1) == 0 ? &kfull[chunk_of(t, v) & 1] : nullptr;
      };
      auto kpar = [&](int v) {
        return (uint32_t)((chunk_of(t, v) >> 1) & 1);
      };
      // two steps of scores ahead; then per step the product with V and the
      // scores of the step after next, into the buffer P just left
      bool ok = wait3(qfull, 0, kbar(0), kpar(0), nullptr, 0);
      if (ok && nv > 0) {
        tc_fence_after();
        issue_s(0);
        issue_s(1);
      }
      for (int v = 0; ok && v < nv; ++v) {
        const int i = chunk_of(t, v), st = i & 1, buf = v & 1;
        ok = wait3(&pfull[2 * t + buf], (v >> 1) & 1,
                   buf == 0 ? &vfull[st] : nullptr, (i >> 1) & 1, kbar(v + 2),
                   kpar(v + 2));
        if (!ok) break;
        tc_fence_after();
        const uint64_t bv =
            umma_desc_sw128(v0 + st * C::KV + buf * kS * 128, kHalf, 1024);
#pragma unroll
        for (int kk = 0; kk < kS / 16; ++kk) {
          const uint64_t bo = bv + (uint64_t)((kk * 2048) >> 4);
          const uint32_t acc = (v > 0 || kk > 0) ? 1u : 0u;
          const uint32_t d = tbase + kColO + 128 * t;
          const uint32_t pa = tbase + kColS + 128 * t + kS * buf + kk * 8;
          if constexpr (PAIR)
            umma2_ts_elect(d, pa, bo, idO, acc);
          else
            umma_ts_elect(d, pa, bo, idO, acc);
        }
        commit(&pvdone[t]);
        if (buf == 1) commit(&vempty[st]);
        if (v + 2 < nv) issue_s(v + 2);
      }
      if (!ok) give_up();
      // every MMA issued has completed before the epilogue and the dealloc
      commit(odone);
      mbar_wait(odone, 0);
    }
  }
  tc_fence_before();
  // every read of tensor memory is done (a pair: and every arrival on the
  // other CTA's barriers)
  if constexpr (PAIR)
    cluster_sync();
  else
    __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    if constexpr (PAIR)
      tmem2_dealloc(tbase, 512);
    else
      tmem_dealloc(tbase, 512);
  }
}

// Parts of output row `at` (the same for the warp's lanes), 0 where no
// sequence has it. Reads what the launch before does not write. The row's
// sequence is looked for 32 at a time, up to the list's first descent: a
// bisection would lose rows of a list that descends later on.
__device__ __forceinline__ int merge_parts(const ExtendParams &p, long at,
                                           int lane) {
  if (at >= (long)p.rows * p.n_h) return 0;
  const int row = (int)at / p.n_h, hh = (int)at - row * p.n_h;  // below 2^31
  const int G = p.n_h / p.n_kv;
  int b = row, r0 = row;
  if (p.row_start) {
    b = -1;
    for (int i0 = 0; i0 < p.batch && b < 0; i0 += 32) {
      int x = 0, y = 0;  // an empty sequence past the batch
      if (i0 + lane < p.batch)
        x = p.row_start[i0 + lane], y = p.row_start[i0 + lane + 1];
      const int has = __ffs(__ballot_sync(0xffffffffu, x <= row && row < y));
      const int down = __ffs(__ballot_sync(0xffffffffu, y < x));
      if (down && (!has || down < has)) return 0;
      if (has) {
        b = i0 + has - 1;
        r0 = __shfl_sync(0xffffffffu, x, has - 1);
      }
    }
    if (b < 0) return 0;
  }
  const Seq q = seq_at(p, b);
  if (row >= r0 + q.n) return 0;  // the sequence was skipped
  const Block k =
      block_at(p, q, ((row - r0) * G + hh % G) / p.block_rows, G);
  int c0, c1;
  block_chunks(k, c0, c1);
  return block_parts(p.chunks_per_split, c1 - c0);
}

// Log-sum-exp merge of the blocks that the launch before split over the
// positions: one warp per output row, a float4 a lane, up to 8 parts'
// loads in flight. The row's parts are found while that launch still runs (it
// lets this one start only after its own predecessor has completed).
constexpr int kRowMergeThreads = 256;

__global__ void __launch_bounds__(kRowMergeThreads)
    extend_merge_kernel(const __grid_constant__ ExtendParams p) {
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long at =
      (long)blockIdx.x * (kRowMergeThreads / 32) + (threadIdx.x >> 5);
  const int parts = merge_parts(p, at, lane);
  pdl_wait();
  if (parts <= 1) return;  // written whole, or no sequence's row
  const long n = (long)p.rows * p.n_h;
  float M, W;
  float4 acc;
  quad_merge<1>(p.ws_lse, p.ws_o, 1, kD, 0, lane, parts,
                [&](int i) { return i * n + at; }, M, W, acc);
  const float iw = W == 0.f ? 0.f : 1.f / W;
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * iw, acc.y * iw);
  packed.y = pack_bf16x2(acc.z * iw, acc.w * iw);
  reinterpret_cast<uint2 *>(p.out + at * kD)[lane] = packed;
  if (lane == 0 && p.lse) p.lse[at] = W == 0.f ? -INFINITY : M + logf(W);
}

}  // namespace

template <int CTAS>
static cudaError_t launch_tc_t(const ExtendParams &p, int blocks, int splits,
                               cudaStream_t s) {
  using C = TCfg<CTAS>;
  static bool done[64] = {};
  auto kern = extend_tc_kernel<CTAS>;
  const cudaError_t e = set_smem_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(blocks * p.n_kv * CTAS, splits), dim3(kThreads),
                    C::SMEM, s, CTAS, p);
}

cudaError_t launch_extend_tc(const ExtendParams &p, int blocks, int splits,
                             cudaStream_t s) {
  const cudaError_t e = p.block_rows == kExtendRows
                            ? launch_tc_t<1>(p, blocks, splits, s)
                            : launch_tc_t<2>(p, blocks, splits, s);
  if (e != cudaSuccess || splits <= 1) return e;
  const long rows = (long)p.rows * p.n_h;
  const long per = kRowMergeThreads / 32;
  return launch_pdl(extend_merge_kernel,
                    dim3((unsigned)((rows + per - 1) / per)),
                    dim3(kRowMergeThreads), 0, s, 1, p);
}

}  // namespace kvd
