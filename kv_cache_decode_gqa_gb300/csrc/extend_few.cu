// Attention of few new rows a sequence over an MXFP4 cache: kvd_gqa_extend
// where a kv head serves at most 16 (row, query head) pairs -- single tokens,
// or a few speculated ones.
//
// A position costs 144 bytes a kv head (72 of K, 72 of V) and 2 x 128
// multiply-adds a pair, so HBM bounds it (6.2 cycles a position and SM) as
// long as the 256 codes of a position are widened in that time. Warp-level
// MMAs (m16n8k16, f16) take K and V straight from registers, with the pairs
// on the other operand in tiles of 8:
//  * S^T = K Q^T, 16 tokens on M, 8 pairs on N. Lane (qr, qc) holds tokens
//    qr and qr + 8 and, over the 8 k-steps, the 32 dims [32 qc, 32 qc + 32):
//    16 bytes of codes and 2 scales a token, two 8-byte loads. A dot product
//    does not depend on the order of its terms, so the query fragments take
//    the same order of dims.
//  * O^T = V^T P^T, 16 dims on M, 8 pairs on N: P^T is the score fragment,
//    packed to f16 and transposed by two movmatrix. Lane (qr, qc) holds
//    columns [16 qr, 16 qr + 16) of tokens 2 qc, 2 qc + 1, 2 qc + 8,
//    2 qc + 9: one scale group a token. The fragment wants pairs of tokens,
//    so the nibbles of two tokens' codes are put together first and one
//    conversion widens the pair.
// So the widening does not grow with the pairs, and pairs beyond 8 cost only
// their products and exponentials. (With O = P V, pairs on M = 16, and the
// maxima reduced every chunk, decode at 8 pairs took 806 instructions per 16
// tokens and ran at a fifth of HBM's rate.) At 32 pairs the tcgen05 kernel is
// ahead (16 sequences of 4 rows and 8 heads a group over 9,200 positions: 102
// us there, 194 us with four tiles of pairs here).
//
// Measured: 32 single tokens, 8 kv heads of 8 pairs over 4,600 positions
// (171 MB), 46 us (the first bytes arrive after 6, the merge launch takes 5);
// 4 kv heads of 16 pairs over 18,400 positions (341 MB), 107 us (with no work
// on them the copies took 72: the widening, products and exponentials of 8
// warps bind it; 16 warps spill with two tiles of pairs, 12 took 5% longer).
//
// A code times its E4M3 scale is exact in f16 (6 significand bits). Queries
// are bf16; each (row, head) is scaled by a power of two so that its largest
// magnitude lies in [2^14, 2^15), which makes the conversion to f16 exact
// except for elements 2^-29 of the largest and below, and is undone in the
// fp32 softmax scale. Scores, references and sums are fp32. Exponentials are
// taken against a reference per pair that moves only when a score passes it
// by 2^(7 + 8) (then the accumulators are rescaled, the reference set 2^7 below
// the maximum, and only then are maxima shared between lanes): they stay below
// 2^15 and the largest is at least 2^7. f16 rounds them by 2^-11, 1/8 of the
// bf16 output's rounding, and drops those 2^-32 of the largest and below (a
// million of them hold 2^-12 of the weight; with the reference at the maximum
// it was 2^-25, and 3%).
//
// Work is split as in the other dense decode kernels (stream_k.cuh): one CTA
// per SM with an equal share of all chunks (and of p.gap empty ones a unit
// where the shares are long), a producer warp that keeps a ring of chunks in
// flight with bulk copies, W consumer warps, and a merge launch for the units
// that CTAs share.
#include <algorithm>
#include <cmath>

#include "prompt_common.cuh"

namespace kvd {
namespace {

constexpr int kD = 128;
constexpr int kRow = 72;  // bytes of a cached row
constexpr int kConsBar = 1;    // named barrier of the consumers
constexpr float kHead = 7.f;   // log2 units a reference lies below the maximum
constexpr float kSlack = 8.f;  // and may lag by

// HP kv heads and CH positions a chunk, RT tiles of 8 pairs, W warps.
template <int HP, int CH, int RT, int W>
struct FCfg {
  static constexpr int THREADS = (W + 1) * 32;  // + the producer warp
  static constexpr int WPH = W / HP;        // consumer warps per kv head
  static constexpr int TPW = CH / WPH;      // tokens per warp and chunk
  static constexpr int NSUB = TPW / 16;
  static constexpr int PAIRS = 8 * RT;      // pair slots of a kv head
  static constexpr int GU = HP * PAIRS;     // pair slots of a unit
  static constexpr int STAGE = HP * CH * kRow;  // K (or V) of a chunk
  // With 16 warps a thread has 96 registers: one chain of score products and
  // V's loads behind them then win over two chains and early loads.
  static constexpr bool LEAN = W == 16;
  // flush slot: 8 * SR pairs of every warp's state at a time
  static constexpr int SR = W * RT > 16 ? 16 / W : RT;
  static constexpr int SLOT = W * 8 * SR * (kD + 2);  // floats
  static constexpr int QF = HP * 8 * RT * 32 * 8;  // query fragments:
                                                   // [head][k][tile][lane]
  static constexpr int FIXED =
      SLOT * 4 + QF + (int)sizeof(WorkPartition) + 64 + 2 * 16 * 8;
  // (223 KB: a merge CTA fits beside this one)
  static constexpr int NS_FIT = (223 * 1024 - FIXED) / (2 * STAGE);
  static constexpr int NS = NS_FIT > W ? W : NS_FIT;
  static constexpr int SLOT_OFF = 2 * NS * STAGE;
  static constexpr int QF_OFF = SLOT_OFF + SLOT * 4;
  static constexpr int WP_OFF = QF_OFF + QF;
  static constexpr int BAR_OFF =
      (WP_OFF + (int)sizeof(WorkPartition) + 15) / 16 * 16;
  static constexpr int SMEM = BAR_OFF + 2 * NS * 8;
  static_assert(TPW % 16 == 0 && NS >= 2 && SMEM <= 223 * 1024, "shape");
};

// An 8 x 8 matrix of 16-bit elements, a row a quad of lanes, transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(r)
               : "r"(x));
  return r;
}

template <int HP, int CH, int RT, int W>
__global__ void __launch_bounds__(FCfg<HP, CH, RT, W>::THREADS, 1)
    extend_few_kernel(const __grid_constant__ ExtendParams p) {
  using C = FCfg<HP, CH, RT, W>;
  constexpr int kConsumers = W * 32;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *sk = smem;
  uint8_t *sv = smem + C::NS * C::STAGE;
  float *slot = reinterpret_cast<float *>(smem + C::SLOT_OFF);
  WorkPartition &wp = *reinterpret_cast<WorkPartition *>(smem + C::WP_OFF);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
  uint64_t *empty = full + C::NS;
  __shared__ int s_len_err, s_list_end;
  __shared__ volatile int s_abort, s_issued, s_producer_done;

  const int G = p.n_h / p.n_kv;
  const int n_units = p.n_kv / HP;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();  // after the wait: the merge launch never overlaps this
                  // launch's predecessor
  if (tid == 0) {
    s_len_err = 0;
    s_abort = 0;
    s_issued = 0;
    s_producer_done = 0;
  }
  __syncthreads();
  build_rows_partition(wp, p, &s_len_err, &s_list_end, CH, n_units, p.gap);
  const int total = wp.total;
  const int P = p.whole_units ? (int)gridDim.x
                              : min((int)gridDim.x, max(total, 1));
  const int c = blockIdx.x;
  // the rows that see nothing (spread over the CTAs by sequence), and the
  // flags of bad lengths and row lists
  for (int b = c; b < p.batch; b += gridDim.x) {
    const int n = b < s_list_end ? seq_rows(p, b) : 0;
    if (tid == 0 && p.row_start && n == 0 &&
        p.row_start[b] != p.row_start[b + 1])
      report(p.err, DEVERR_LEN);
    if (wp.nch[b] != 0) continue;
    const long row0 = p.row_start ? p.row_start[b] : b;
    for (int i = tid; i < n * p.n_h * (kD / 8); i += C::THREADS)
      reinterpret_cast<uint4 *>(p.out + row0 * p.n_h * kD)[i] =
          make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = tid; i < n * p.n_h; i += C::THREADS)
        p.lse[row0 * p.n_h + i] = -INFINITY;
  }
  if (c == 0 && tid == 0 && s_len_err) report(p.err, DEVERR_LEN);
  if (c >= P || total == 0) return;
  const int lo = p.whole_units ? unit_lo(wp, p.batch, n_units, c)
                               : range_lo(c, total, P);
  const int hi = p.whole_units ? unit_lo(wp, p.batch, n_units, c + 1)
                               : range_lo(c + 1, total, P);
  const int n = hi - lo;
  if (n == 0) return;

  if (tid == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], W);
    }
    fence_mbar_init();
  }
  __syncthreads();

  // ======================= producer warp ==================================
  if (warp == W) {
    const uint64_t policy = policy_evict_first();
    const int bs = p.block_size;
    auto block_of = [&](int b, int lb) {
      int pb = p.block_table[(long)b * p.max_blocks + lb];
      if (pb < 0 || pb >= p.num_blocks) {
        report(p.err, DEVERR_BLOCK);
        pb = 0;  // read a valid block; the result is flagged as wrong
      }
      return pb;
    };
    // Chunks are looked up 32 / L at a time: lane l takes block l % L of
    // chunk l / L of the batch (L: blocks a chunk may touch, a power of
    // two), and later issues that block's copies. Attended positions are
    // widened to even bounds (rows of 72 bytes are copied in pairs; block
    // sizes are even). L > 32 (blocks of 2 .. 8 positions): a lane takes
    // further blocks when it issues.
    int L = 1;
    while (L < 32 && L < (bs % CH == 0   ? 1
                          : CH % bs == 0 ? CH / bs
                                         : CH / bs + 2))
      L <<= 1;
    const int q = lane & (L - 1), batch = 32 / L;
    int s = 0, ph = 1;  // a fresh barrier passes a wait for parity 1
    int used = 0;       // stages filled so far
    bool go = true;
    for (int base = 0; go && base < n; base += batch) {
      const int mine = base + lane / L;
      int tok = 0, t0 = 0, t1 = 0, b0 = 0, nb = 0, pb = 0;
      ChunkCursor cur{0, 0, 0};
      if (mine < n) cur = cursor_at(wp, p.batch, lo + mine);
      const bool empty_chunk =
          mine >= n || cur.k >= wp.nch[cur.b] - p.gap;
      if (!empty_chunk) {
        const int len = wp.len[cur.b];
        tok = rows_first(p, cur.b, len, CH) + cur.k * CH;
        t0 = max(tok, rows_lo(p, cur.b, len)) & ~1;
        t1 = (min(tok + CH, len) + 1) & ~1;
        b0 = t0 / bs;
        nb = (t1 - 1) / bs - b0 + 1;
        if (q < nb) pb = block_of(cur.b, b0 + q);
      }
      const int cnt = min(batch, n - base);
      for (int j = 0; j < cnt; ++j) {
        if (__shfl_sync(0xffffffffu, empty_chunk, j * L)) continue;
        go = mbar_wait(&empty[s], ph);
        if (!go) report(p.err, DEVERR_TIMEOUT);
        go = __all_sync(0xffffffffu, go && !s_abort);
        if (!go) break;
        if (lane == j * L) {
          mbar_arrive_expect_tx(&full[s], 2u * HP * (t1 - t0) * kRow);
          s_issued = used + 1;
        }
        ++used;
        __syncwarp();
        if (lane / L == j) {
          for (int k = q; k < nb; k += L) {
            if (k >= L) pb = block_of(cur.b, b0 + k);
            const int lb = (b0 + k) * bs;
            // (a last block may end past 2^31)
            const int a0 = max(t0, lb), a1 = (int)min((long)t1, (long)lb + bs);
            const long row = ((long)pb * p.n_kv + cur.h * HP) * bs + (a0 - lb);
            const int off = s * C::STAGE + (a0 - tok) * kRow;
            // whole blocks of a chunk's length hold the unit's heads side by
            // side
            const bool joined = HP > 1 && bs == CH && a1 - a0 == CH;
            const uint32_t bytes =
                (uint32_t)(a1 - a0) * kRow * (joined ? HP : 1);
            const int heads = joined ? 1 : HP;
            for (int g = 0; g < heads; ++g) {
              const long src = (row + (long)g * bs) * kRow;
              bulk_g2s_hint(sk + off + g * CH * kRow, p.k + src, bytes,
                            &full[s], policy);
              bulk_g2s_hint(sv + off + g * CH * kRow, p.v + src, bytes,
                            &full[s], policy);
            }
          }
        }
        __syncwarp();
        if (++s == C::NS) s = 0, ph ^= 1;
      }
    }
    __syncwarp();
    if (lane == 0) s_producer_done = 1;
    return;
  }

  // ======================= consumer warps =================================
  // Pair slot j of a kv head: the sequence's row j / G, query head j % G of
  // the head's group. In the score and output fragments lane (qr, qc) holds
  // pairs 8 r + 2 qc and 8 r + 2 qc + 1; of the scores tokens qr and qr + 8,
  // of the outputs dims [16 qr, 16 qr + 16). Query fragments are of pair 8 r
  // + qr.
  const int qr = lane >> 2, qc = lane & 3;
  const int hj = warp / C::WPH;              // kv head of the unit
  const int wt0 = (warp % C::WPH) * C::TPW;  // this warp's first token
  uint2 *qf = reinterpret_cast<uint2 *>(smem + C::QF_OFF) + hj * 8 * RT * 32;
  float o[RT][8][4];
  // per pair 8 r + 2 qc + q: the reference (0 before the first score, when
  // `none` is set), the sum over this lane's tokens, the scores' scale
  float ref[RT][2], l[RT][2], sl[RT][2];
  bool none[RT][2];
  int ulo = 0, un = 0, T = 0;
  long urow = 0;
  bool ok = true;

  // positions [lo, hi) that pair slot j sees
  auto pair_range = [&](int b, int j, int &lo_, int &hi_) {
    const int t = j / G, pos = T - un + t;
    const int s_b = p.win_start ? max(p.win_start[b], 0) : 0;
    lo_ = p.window > 0 ? max(s_b, window_lo(p, pos)) : s_b;
    hi_ = t < un ? max(pos + 1, 0) : 0;
  };

  auto start_unit = [&](int b, int h) {
    T = wp.len[b];
    un = seq_rows(p, b);
    urow = p.row_start ? p.row_start[b] : b;
    ulo = rows_lo(p, b, T);
    const int kvh = h * HP + hj;
    // (every warp of a head writes the same query fragments; finish_unit's
    // barriers keep them apart from the last unit's readers)
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int j = qr + 8 * r, t = j / G, g = j - t * G;
      const bool live = t < un;
      uint4 x[4];
      uint32_t m = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x[v] = make_uint4(0, 0, 0, 0);
        if (live)
          x[v] = *reinterpret_cast<const uint4 *>(
              p.q + (urow + t) * p.q_rs + ((long)kvh * G + g) * p.q_hs +
              32 * qc + 8 * v);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        m = __vmaxu2(m, __vmaxu2(x[v].x & 0x7fff7fffu, x[v].y & 0x7fff7fffu));
        m = __vmaxu2(m, __vmaxu2(x[v].z & 0x7fff7fffu, x[v].w & 0x7fff7fffu));
      }
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = row_exponent(m);
      const float f = __uint_as_float((uint32_t)e << 23);
      const float sc =
          fmaxf(p.scale_log2 * exp2f((float)(127 - e)), 1.17549435e-38f);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        sl[r][q] = __shfl_sync(0xffffffffu, sc, 8 * qc + 4 * q);
        ref[r][q] = 0.f;
        none[r][q] = true;
        l[r][q] = 0.f;
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t w[4] = {x[v].x, x[v].y, x[v].z, x[v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t y = pack_f16x2(bf16lo(w[k]) * f, bf16hi(w[k]) * f);
          const int kk = 2 * v + (k >> 1);
          reinterpret_cast<uint32_t *>(qf + (kk * RT + r) * 32 +
                                       lane)[k & 1] = y;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[r][i][q] = 0.f;
    }
    named_sync(kConsBar, kConsumers);  // the fragments are written
  };

  // Every warp's state of the unit through the slot (SR tiles of pairs at a
  // time), then its pairs as outputs (a unit wholly in this CTA's range) or
  // as this CTA's partial of it: M = max m_w, L = sum l_w 2^(m_w - M), out =
  // sum_w 2^(m_w - M) o_w / L.
  auto finish_unit = [&](int b, int h) {
    constexpr int SP = 8 * C::SR;  // pairs a round
    float *wm = slot;              // [warp][SP]
    float *wl = wm + W * SP;       // [warp][SP]
    float *wo = wl + W * SP;       // [warp][SP][D]
    const int ustart = wp.pre[b] + h * wp.nch[b];
    const int uend = ustart + wp.nch[b] - p.gap;
    const bool whole = ustart >= lo && uend <= hi;
    const long wslot = c * 2 + partial_side(ustart, lo);
    const int pairs = un * G;
#pragma unroll
    for (int r0 = 0; r0 < RT; r0 += C::SR) {
      named_sync(kConsBar, kConsumers);  // the slot is free
#pragma unroll
      for (int rr = 0; rr < C::SR; ++rr) {
        const int r = r0 + rr;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float t = l[r][q];  // over the lanes of all tokens
          t += __shfl_xor_sync(0xffffffffu, t, 4);
          t += __shfl_xor_sync(0xffffffffu, t, 8);
          t += __shfl_xor_sync(0xffffffffu, t, 16);
          if (qr == 0) {
            wm[warp * SP + 8 * rr + 2 * qc + q] =
                none[r][q] ? -INFINITY : ref[r][q];
            wl[warp * SP + 8 * rr + 2 * qc + q] = t;
          }
          float *dst = wo + (warp * SP + 8 * rr + 2 * qc + q) * kD + 16 * qr;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            reinterpret_cast<float4 *>(dst)[v] =
                make_float4(o[r][2 * v][q], o[r][2 * v][2 + q],
                            o[r][2 * v + 1][q], o[r][2 * v + 1][2 + q]);
        }
      }
      named_sync(kConsBar, kConsumers);
      const int rows = min(max(pairs - 8 * r0, 0), SP);  // of this round
      for (int jg = warp; jg < HP * rows; jg += W) {
        const int j = jg / rows, g = jg - j * rows, w0 = j * C::WPH;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::WPH; ++w) M = fmaxf(M, wm[(w0 + w) * SP + g]);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < C::WPH; ++w) {
          const float mw = wm[(w0 + w) * SP + g];
          const float cw = mw == -INFINITY ? 0.f : ex2(mw - M);
          L = fmaf(wl[(w0 + w) * SP + g], cw, L);
          const float4 v = reinterpret_cast<const float4 *>(
              wo + ((w0 + w) * SP + g) * kD)[lane];
          acc.x = fmaf(cw, v.x, acc.x);
          acc.y = fmaf(cw, v.y, acc.y);
          acc.z = fmaf(cw, v.z, acc.z);
          acc.w = fmaf(cw, v.w, acc.w);
        }
        // a NaN among a pair's scores stays one: its L is NaN
        const float f = L == 0.f ? 0.f : 1.f / L;
        acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
        const float lse = L == 0.f ? -INFINITY
                                   : (M + log2f(L)) * 0.69314718055994531f;
        const int pair = 8 * r0 + g;
        if (whole) {
          const long at = (urow + pair / G) * p.n_h +
                          (long)(h * HP + j) * G + pair % G;
          uint2 packed;
          packed.x = pack_bf16x2(acc.x, acc.y);
          packed.y = pack_bf16x2(acc.z, acc.w);
          reinterpret_cast<uint2 *>(p.out + at * kD)[lane] = packed;
          if (lane == 0 && p.lse) p.lse[at] = lse;
        } else {
          const long at = wslot * C::GU + j * C::PAIRS + pair;
          reinterpret_cast<float4 *>(p.ws_o + at * kD)[lane] = acc;
          if (lane == 0) p.ws_lse[at] = lse;
        }
      }
    }
  };

  int s = 0, ph = 0;
  for (int x = lo; x < hi;) {
    const ChunkCursor cc = cursor_at(wp, p.batch, x);
    const int left = wp.nch[cc.b] - cc.k;  // of the unit, empty ones with it
    const int nk = min(left - p.gap, hi - x);
    x += left;
    if (nk <= 0) continue;
    start_unit(cc.b, cc.h);
    int ctok = rows_first(p, cc.b, T, CH) + cc.k * CH;
    // positions that every pair sees; others are masked pair by pair
    const int all_lo =
        max(p.win_start ? max(p.win_start[cc.b], 0) : 0,
            p.window > 0 ? T - p.window : 0);
    const int all_hi = T - un + 1;
    for (int i = 0; i < nk; ++i, ctok += CH) {
      if (ok && !(ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ph))) &&
          lane == 0) {
        report(p.err, DEVERR_TIMEOUT);
        s_abort = 1;
      }
      const uint8_t *kl = sk + s * C::STAGE + (hj * CH + wt0 + qr) * kRow;
      const uint8_t *vl =
          sv + s * C::STAGE + (hj * CH + wt0 + 2 * qc) * kRow + 8 * qr;
#pragma unroll 1
      for (int u = 0; u < (ok ? C::NSUB : 0); ++u) {
        const int pos0 = ctok + wt0 + 16 * u;  // the tile's first position
        const uint8_t *kr = kl + u * 16 * kRow;
        const uint8_t *vr = vl + u * 16 * kRow;
        // V's codes and scales: on their way during the scores, or (LEAN)
        // behind them
        uint2 v0[2], v1[2];  // tokens 2 qc + 8 t and the next
        uint32_t vs[2];
        const bool outside = pos0 < ulo || pos0 + 16 > T;
        auto load_v = [&]() {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint8_t *row = vr + 8 * t * kRow;
            v0[t] = *reinterpret_cast<const uint2 *>(row);
            v1[t] = *reinterpret_cast<const uint2 *>(row + kRow);
            uint32_t a = row[64 - 7 * qr], z = row[kRow + 64 - 7 * qr];
            if (outside) {
              // rows outside the unit's positions were not copied: their
              // scales are taken as 0, so that 0 times them stays 0
              const int pos = pos0 + 8 * t + 2 * qc;
              if (pos < ulo || pos >= T) a = 0;
              if (pos + 1 < ulo || pos + 1 >= T) z = 0;
            }
            vs[t] = a | (z << 8);
          }
        };
        if constexpr (!C::LEAN) load_v();
        // ---- S^T = K Q^T of 16 tokens (two chains of products, or one) ----
        float sc[RT][4], sd[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) sc[r][q] = sd[r][q] = 0.f;
        {
          uint32_t w[2][4], s0[2], s1[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint8_t *row = kr + 8 * t * kRow;
            const uint2 c0 = *reinterpret_cast<const uint2 *>(row + 16 * qc);
            const uint2 c1 =
                *reinterpret_cast<const uint2 *>(row + 16 * qc + 8);
            const uint32_t sp = e4m3x2_to_f16x2(
                *reinterpret_cast<const uint16_t *>(row + 64 + 2 * qc));
            s0[t] = prmt(sp, 0, 0x1010), s1[t] = prmt(sp, 0, 0x3232);
            w[t][0] = c0.x, w[t][1] = c0.y, w[t][2] = c1.x, w[t][3] = c1.y;
          }
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            uint32_t y[2][4];
            e2m1x8_to_f16(w[0][k4], y[0]);
            e2m1x8_to_f16(w[1][k4], y[1]);
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              const uint32_t a[4] = {
                  mul_f16x2(y[0][2 * h2], k4 < 2 ? s0[0] : s1[0]),
                  mul_f16x2(y[1][2 * h2], k4 < 2 ? s0[1] : s1[1]),
                  mul_f16x2(y[0][2 * h2 + 1], k4 < 2 ? s0[0] : s1[0]),
                  mul_f16x2(y[1][2 * h2 + 1], k4 < 2 ? s0[1] : s1[1])};
#pragma unroll
              for (int r = 0; r < RT; ++r) {
                const uint2 f = qf[((2 * k4 + h2) * RT + r) * 32 + lane];
                mma_f16(h2 && !C::LEAN ? sd[r] : sc[r], a, f.x, f.y);
              }
            }
          }
        }
        if constexpr (!C::LEAN) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) sc[r][q] += sd[r][q];
        }
        // ---- exponentials (q: pair q % 2, token qr + 8 (q / 2)) ----
        bool grow = false;
        if (pos0 < all_lo || pos0 + 16 > all_hi) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              int vlo, vhi;
              pair_range(cc.b, 8 * r + 2 * qc + q, vlo, vhi);
              const int pa = pos0 + qr, pz = pos0 + qr + 8;
              if (pa < vlo || pa >= vhi) sc[r][q] = -INFINITY;
              if (pz < vlo || pz >= vhi) sc[r][2 + q] = -INFINITY;
            }
        }
        // exponents against the references; a first score, or one past its
        // reference by kHead + kSlack, moves them
        float t[RT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            t[r][q] = fmaf(sc[r][q], sl[r][q & 1], -ref[r][q & 1]);
            grow |= t[r][q] > (none[r][q & 1] ? -INFINITY : kHead + kSlack);
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float m = fmaxf(sc[r][q], sc[r][2 + q]) * sl[r][q] - kHead;
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              if (!none[r][q]) m = fmaxf(m, ref[r][q]);
              if (m == -INFINITY) continue;  // still no score (or all NaN)
              const float f = none[r][q] ? 0.f : ex2(ref[r][q] - m);
              ref[r][q] = m;
              l[r][q] *= f;
#pragma unroll
              for (int d = 0; d < 8; ++d) {
                o[r][d][q] *= f;
                o[r][d][2 + q] *= f;
              }
              none[r][q] = false;
              t[r][q] = fmaf(sc[r][q], sl[r][q], -m);
              t[r][2 + q] = fmaf(sc[r][2 + q], sl[r][q], -m);
            }
        }
        uint32_t pb[RT][2];  // P^T fragments
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float e0 = ex2(t[r][0]), e1 = ex2(t[r][1]);
          const float e2 = ex2(t[r][2]), e3 = ex2(t[r][3]);
          l[r][0] += e0 + e2;
          l[r][1] += e1 + e3;
          pb[r][0] = transpose_8x8(pack_f16x2(e0, e1));
          pb[r][1] = transpose_8x8(pack_f16x2(e2, e3));
        }
        // ---- O^T += V^T P^T ----
        if constexpr (C::LEAN) load_v();
        uint32_t e[2][2], d[2][2];  // [token pair][word]: even, odd dims
        uint32_t sp[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          sp[t] = e4m3x2_to_f16x2((uint16_t)vs[t]);
          e[t][0] = (v0[t].x & 0x0f0f0f0fu) | ((v1[t].x << 4) & 0xf0f0f0f0u);
          e[t][1] = (v0[t].y & 0x0f0f0f0fu) | ((v1[t].y << 4) & 0xf0f0f0f0u);
          d[t][0] = ((v0[t].x >> 4) & 0x0f0f0f0fu) | (v1[t].x & 0xf0f0f0f0u);
          d[t][1] = ((v0[t].y >> 4) & 0x0f0f0f0fu) | (v1[t].y & 0xf0f0f0f0u);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t x2[2][4], y2[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            e2m1x8_to_f16(e[t][w], x2[t]);
            e2m1x8_to_f16(d[t][w], y2[t]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // M tile: dims 16 qr + 2 (4 w + k) (rows qr) and + 1 (qr + 8)
            const uint32_t a[4] = {
                mul_f16x2(x2[0][k], sp[0]), mul_f16x2(y2[0][k], sp[0]),
                mul_f16x2(x2[1][k], sp[1]), mul_f16x2(y2[1][k], sp[1])};
#pragma unroll
            for (int r = 0; r < RT; ++r)
              mma_f16(o[r][4 * w + k], a, pb[r][0], pb[r][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == C::NS) s = 0, ph ^= 1;
    }
    finish_unit(cc.b, cc.h);
  }
  if (s_abort && tid == 0) {
    // after an abort: every copy that was issued has landed before this CTA
    // gives its shared memory back
    for (int t = 0; t < (1 << 20) && !s_producer_done; ++t) __nanosleep(1000);
    const int issued = s_issued;
    for (int st = 0; st < C::NS; ++st) {
      int last = -1;
      for (int c2 = st; c2 < issued; c2 += C::NS) last = c2;
      if (last >= 0) mbar_wait(&full[st], (last / C::NS) & 1);
    }
  }
}

// Log-sum-exp merge of the units that several CTAs of the launch before
// share, up to 8 parts' loads of a float4 in flight a lane: one warp a pair,
// or (LANES = 4, units of many parts) four lanes a float4 and a CTA a pair.
// A CTA is small enough to sit beside one of
// that launch (128 threads, 64 registers, 1 KB for batches up to 64), so
// that the partition is rebuilt while it still runs, and takes every
// gridDim.x-th group of pairs; eight fit an SM (two an SM: 3 to 4 us more for
// 2,048 pairs). (256 threads and a CTA per two pairs started only when the
// other launch had left the SMs: 10 us in all for 32 sequences of 8 kv
// heads.)
constexpr int kRowMergeThreads = 128;

template <int NB, int LANES>
__global__ void __launch_bounds__(kRowMergeThreads, 8)
    merge_few_kernel(const __grid_constant__ ExtendParams p, int n_units,
                     int hp, int chunk, int slots) {
  __shared__ WorkPartitionT<NB> wp;
  __shared__ int s_len_err, s_list_end;
  pdl_trigger();
  // the lengths and row lists are read before the launch before completes:
  // it does not write them, and it lets this one start only after its own
  // predecessor has completed
  build_rows_partition(wp, p, &s_len_err, &s_list_end, chunk, n_units, p.gap);
  pdl_wait();
  const int total = wp.total;
  if (total == 0) return;
  const int P = min(p.n_splits, total);
  const int G = p.n_h / p.n_kv;
  const int gu = hp * slots;  // pair slots of a unit
  const int per_head = min(slots, p.max_rows * G);
  const int per_unit = hp * per_head;
  constexpr int PAIR_THREADS = 32 * LANES, PAIRS = kRowMergeThreads /
                                                  PAIR_THREADS;
  const int x = threadIdx.x % PAIR_THREADS, e4 = x / LANES;
  const int step = gridDim.x * PAIRS;
  const int items = p.batch * n_units * per_unit;
  for (int it = blockIdx.x * PAIRS + threadIdx.x / PAIR_THREADS; it < items;
       it += step) {
    const int u = it / per_unit, jg = it - u * per_unit;
    const int j = jg / per_head, g = jg - j * per_head;
    const int b = u / n_units, h = u - b * n_units;
    if (wp.nch[b] == 0 || g >= seq_rows(p, b) * G) continue;
    const int ustart = wp.pre[b] + h * wp.nch[b];
    const int c_first = cta_of(ustart, total, P);
    const int parts =
        cta_of(ustart + wp.nch[b] - p.gap - 1, total, P) - c_first + 1;
    if (parts == 1) continue;
    const long row0 = p.row_start ? p.row_start[b] : b;
    const int sl = j * slots + g;
    float M, W;
    float4 acc;
    quad_merge<LANES>(p.ws_lse, p.ws_o, gu, kD, sl, sl * (kD / 4) + e4, parts,
                      [&](int i) {
                        return (long)(c_first + i) * 2 + (i == 0 ? 1 : 0);
                      },
                      M, W, acc);
    if (x % LANES != 0) continue;
    const float iw = W == 0.f ? 0.f : 1.f / W;
    const long at = (row0 + g / G) * p.n_h + (long)(h * hp + j) * G + g % G;
    uint2 packed;
    packed.x = pack_bf16x2(acc.x * iw, acc.y * iw);
    packed.y = pack_bf16x2(acc.z * iw, acc.w * iw);
    reinterpret_cast<uint2 *>(p.out + at * kD)[e4] = packed;
    if (e4 == 0 && p.lse)
      p.lse[at] = W == 0.f ? -INFINITY : M + logf(W);
  }
}

template <int HP, int CH, int RT, int W>
cudaError_t launch_few_t(const ExtendParams &p, cudaStream_t s) {
  using C = FCfg<HP, CH, RT, W>;
  auto kern = extend_few_kernel<HP, CH, RT, W>;
  static bool done[64] = {};
  cudaError_t e = set_smem_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(p.n_splits), dim3(C::THREADS), C::SMEM, s, 1, p);
  if (e != cudaSuccess || p.whole_units || p.n_splits <= 1) return e;
  const int n_units = p.n_kv / HP;
  const long pairs = (long)p.batch * n_units * HP *
                     std::min(C::PAIRS, p.max_rows * (p.n_h / p.n_kv));
  // parts of a unit of average length
  const bool many = p.n_splits > 6L * p.batch * n_units;
  const long per = many ? 1 : kRowMergeThreads / 32;
  const dim3 grid((unsigned)std::min((pairs + per - 1) / per, 1216L));
  auto merge = p.batch <= kMergeSmallBatch
                   ? (many ? merge_few_kernel<kMergeSmallBatch, 4>
                           : merge_few_kernel<kMergeSmallBatch, 1>)
                   : (many ? merge_few_kernel<kMaxDecodeBatch, 4>
                           : merge_few_kernel<kMaxDecodeBatch, 1>);
  return launch_pdl(merge, grid, dim3(kRowMergeThreads), 0, s, 1, p, n_units,
                    HP, CH, C::PAIRS);
}

template <int HP, int CH, int W1, int W2>
cudaError_t launch_few_rt(const ExtendParams &p, int tiles, cudaStream_t s) {
  return tiles == 1 ? launch_few_t<HP, CH, 1, W1>(p, s)
                    : launch_few_t<HP, CH, 2, W2>(p, s);
}

}  // namespace

// Large chunks (256 (position, head) rows: 37 KB) keep the copies large;
// small ones (128) spread a little work over more CTAs. Where a block holds
// 64 positions, its heads lie side by side and one copy moves several.
FewPlan extend_few_plan(int n_kv, int block_size, int pairs, long batch,
                        int max_seq_len, int sms) {
  FewPlan f;
  f.tiles = pairs <= 8 ? 1 : 2;
  const bool large =
      batch * n_kv * (((long)max_seq_len + 255) / 256) >= 4L * sms;
  if (large) {
    f.hp = block_size == 64 && n_kv % 4 == 0 ? 4 : 1;
    f.chunk = 256 / f.hp;
  } else {
    f.hp = block_size == 64 && n_kv % 2 == 0 ? 2 : 1;
    f.chunk = 128 / f.hp;
  }
  return f;
}

cudaError_t launch_extend_few(const ExtendParams &p, const FewPlan &f,
                              cudaStream_t s) {
  if (p.batch > kMaxDecodeBatch) return cudaErrorNotSupported;
  switch (f.hp * 1000 + f.chunk) {
    case 4064: return launch_few_rt<4, 64, 16, 8>(p, f.tiles, s);
    case 1256: return launch_few_rt<1, 256, 16, 8>(p, f.tiles, s);
    case 2064: return launch_few_rt<2, 64, 8, 8>(p, f.tiles, s);
    default: return launch_few_rt<1, 128, 8, 8>(p, f.tiles, s);
  }
}

}  // namespace kvd
