// Attention of few new rows a sequence over an MXFP4 cache: kvd_gqa_extend
// where a kv head serves at most 16 (row, query head) pairs -- single tokens
// of query groups up to 16, or a few speculated tokens of smaller groups.
//
// A position costs 144 bytes a kv head (72 of K, 72 of V) and 2 x 16 x 128
// multiply-adds, so HBM bounds it as long as the 256 codes of a position are
// widened fast enough. The warp-level MMA m16n8k16 takes the rows on M = 16,
// and both operands are widened straight into its fragments:
//  * K: lane (qr, qc) of the fragment holds token qr and, over the 8 k-steps,
//    the 32 dims [32 qc, 32 qc + 32): 16 bytes of codes and 2 scales, read
//    with two 8-byte loads. A dot product does not depend on the order of
//    its terms, so the query fragments take the same order of dims.
//  * V: lane (qr, qc) holds columns [16 qr, 16 qr + 16) of tokens 2 qc,
//    2 qc + 1, 2 qc + 8, 2 qc + 9: one scale group a token. The fragment
//    wants pairs of tokens, so the nibbles of two tokens' codes are put
//    together first and one conversion widens the pair.
// A code times its E4M3 scale is exact in f16 (6 significand bits). Queries
// are bf16; each (row, head) is scaled by a power of two so that its largest
// magnitude lies in [2^14, 2^15), which makes the conversion to f16 exact
// except for elements 2^-29 of the largest and below, and is undone in the
// fp32 softmax scale. Scores, running maxima and sums are fp32.
// Probabilities are at most 1 and enter the second product as f16 (relative
// rounding 2^-11, 1/8 of the bf16 output's).
//
// Work is split as in the other dense decode kernels (stream_k.cuh): one CTA
// per SM with an equal share of all chunks, a producer warp that keeps a
// ring of chunks in flight with bulk copies, eight consumer warps, and a
// merge launch for the units that CTAs share.
#include <algorithm>
#include <cmath>

#include "kvd_common.cuh"
#include "stream_k.cuh"

namespace kvd {
namespace {

constexpr int kD = 128;
constexpr int kRow = 72;                   // bytes of a cached row
constexpr int kWarps = 8;                  // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kThreads = kConsumers + 32;  // + the producer warp
constexpr int kConsBar = 1;                // named barrier of the consumers

template <int HP, int CH>
struct FCfg {
  static constexpr int WPH = kWarps / HP;   // consumer warps per kv head
  static constexpr int TPW = CH / WPH;      // tokens per warp and chunk
  static constexpr int NSUB = TPW / 16;
  static constexpr int GU = HP * kFewRows;  // row slots of a unit
  static constexpr int STAGE = HP * CH * kRow;  // K (or V) of a chunk
  static constexpr int SLOT = kWarps * kFewRows * (kD + 2);  // floats
  static constexpr int FIXED =
      SLOT * 4 + (int)sizeof(WorkPartition) + 64 + 2 * 16 * 8;
  static constexpr int NS_FIT = (226 * 1024 - FIXED) / (2 * STAGE);
  static constexpr int NS = NS_FIT > 16 ? 16 : NS_FIT;
  static constexpr int SLOT_OFF = 2 * NS * STAGE;
  static constexpr int WP_OFF = SLOT_OFF + SLOT * 4;
  static constexpr int BAR_OFF =
      (WP_OFF + (int)sizeof(WorkPartition) + 15) / 16 * 16;
  static constexpr int SMEM = BAR_OFF + 2 * NS * 8;
  static_assert(TPW % 16 == 0 && NS >= 2 && SMEM <= 226 * 1024, "shape");
};

template <int HP, int CH>
__global__ void __launch_bounds__(kThreads, 1)
    extend_few_kernel(const __grid_constant__ ExtendParams p) {
  using C = FCfg<HP, CH>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t *sk = smem;
  uint8_t *sv = smem + C::NS * C::STAGE;
  float *slot = reinterpret_cast<float *>(smem + C::SLOT_OFF);
  WorkPartition &wp = *reinterpret_cast<WorkPartition *>(smem + C::WP_OFF);
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);
  uint64_t *empty = full + C::NS;
  __shared__ int s_len_err;
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
  build_partition(wp, p, &s_len_err, CH, n_units);
  const int total = wp.total;
  const int P = p.whole_units ? (int)gridDim.x
                              : min((int)gridDim.x, max(total, 1));
  const int c = blockIdx.x;
  // the rows that see nothing (spread over the CTAs by sequence), and the
  // flags of bad lengths and row lists
  for (int b = c; b < p.batch; b += gridDim.x) {
    const int n = seq_rows(p, b);
    if (tid == 0 && p.row_start && n == 0 &&
        p.row_start[b] != p.row_start[b + 1])
      report(p.err, DEVERR_LEN);
    if (wp.nch[b] != 0) continue;
    const long row0 = p.row_start ? p.row_start[b] : b;
    for (int i = tid; i < n * p.n_h * (kD / 8); i += kThreads)
      reinterpret_cast<uint4 *>(p.out + row0 * p.n_h * kD)[i] =
          make_uint4(0, 0, 0, 0);
    if (p.lse)
      for (int i = tid; i < n * p.n_h; i += kThreads)
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
      mbar_init(&empty[s], kWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();

  // ======================= producer warp ==================================
  if (warp == kWarps) {
    const uint64_t policy = policy_evict_first();
    const int bs = p.block_size;
    ChunkCursor cur = cursor_at(wp, p.batch, lo);
    int s = 0, ph = 1;  // a fresh barrier passes a wait for parity 1
    for (int i = 0; i < n; ++i) {
      // the chunk's attended positions [t0, t1), widened to even bounds
      // (rows of 72 bytes are copied in pairs; block sizes are even), and
      // their blocks, one a lane
      const int T = wp.len[cur.b];
      const int tok = seq_first(p, cur.b, T, CH) + cur.k * CH;
      const int t0 = max(tok, seq_lo(p, cur.b, T)) & ~1;
      const int t1 = (min(tok + CH, T) + 1) & ~1;
      const int b0 = t0 / bs, nb = (t1 - 1) / bs - b0 + 1;
      auto block_of = [&](int j) {
        int pb = p.block_table[(long)cur.b * p.max_blocks + b0 + j];
        if (pb < 0 || pb >= p.num_blocks) {
          report(p.err, DEVERR_BLOCK);
          pb = 0;  // read a valid block; the result is flagged as wrong
        }
        return pb;
      };
      int pb = lane < nb ? block_of(lane) : 0;
      bool go = mbar_wait(&empty[s], ph);
      if (!go) report(p.err, DEVERR_TIMEOUT);
      go = __all_sync(0xffffffffu, go && !s_abort);
      if (!go) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[s], 2u * HP * (t1 - t0) * kRow);
        s_issued = i + 1;
      }
      __syncwarp();
      for (int j = lane; j < nb; j += 32) {
        if (j >= 32) pb = block_of(j);  // blocks of 2 .. 4 positions only
        const int lb = b0 + j;
        const int a0 = max(t0, lb * bs), a1 = min(t1, (lb + 1) * bs);
        const long row = ((long)pb * p.n_kv + cur.h * HP) * bs + (a0 - lb * bs);
        const int off = s * C::STAGE + (a0 - tok) * kRow;
        // whole blocks of a chunk's length hold the unit's heads side by side
        const bool joined = HP > 1 && bs == CH && a1 - a0 == CH;
        const uint32_t bytes = (uint32_t)(a1 - a0) * kRow * (joined ? HP : 1);
#pragma unroll
        for (int q = 0; q < HP; ++q) {
          if (joined && q > 0) break;
          const long src = (row + (long)q * bs) * kRow;
          bulk_g2s_hint(sk + off + q * CH * kRow, p.k + src, bytes, &full[s],
                        policy);
          bulk_g2s_hint(sv + off + q * CH * kRow, p.v + src, bytes, &full[s],
                        policy);
        }
      }
      __syncwarp();
      cursor_next(wp, p.batch, n_units, cur);
      if (++s == C::NS) s = 0, ph ^= 1;
    }
    __syncwarp();
    if (lane == 0) s_producer_done = 1;
    return;
  }

  // ======================= consumer warps =================================
  // Lane (qr, qc): rows qr and qr + 8 of the 16 row slots (slot j: the
  // sequence's row j / G, query head j % G of the kv head).
  const int qr = lane >> 2, qc = lane & 3;
  const int hj = warp / C::WPH;              // kv head of the unit
  const int wt0 = (warp % C::WPH) * C::TPW;  // this warp's first token
  uint32_t qa[8][4];
  float o[16][4];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float sl0 = 0.f, sl1 = 0.f;                // scores into log2 units, by row
  int lo0 = 0, hi0 = 0, lo1 = 0, hi1 = 0;    // positions rows qr, qr + 8 see
  int ulo = 0, un = 0;
  long urow = 0;
  int cur_b = -1, cur_h = -1;
  bool ok = true;

  auto start_unit = [&](int b, int h) {
    const int T = wp.len[b];
    un = seq_rows(p, b);
    urow = p.row_start ? p.row_start[b] : b;
    ulo = seq_lo(p, b, T);
    const int kvh = h * HP + hj;
    const int s_b = p.win_start ? max(p.win_start[b], 0) : 0;
    uint4 x[2][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = qr + 8 * r, t = j / G, g = j - t * G;
      const bool live = t < un;
      const int pos = T - un + t;            // this row's position
      const int rhi = live ? max(pos + 1, 0) : 0;
      const int rlo = p.window > 0 ? max(s_b, pos + 1 - p.window) : s_b;
      if (r == 0) lo0 = rlo, hi0 = rhi;
      else lo1 = rlo, hi1 = rhi;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x[r][v] = make_uint4(0, 0, 0, 0);
        if (live)
          x[r][v] = *reinterpret_cast<const uint4 *>(
              p.q + (urow + t) * p.q_rs + ((long)kvh * G + g) * p.q_hs +
              32 * qc + 8 * v);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      uint32_t m = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        m = __vmaxu2(m, x[r][v].x & 0x7fff7fffu);
        m = __vmaxu2(m, x[r][v].y & 0x7fff7fffu);
        m = __vmaxu2(m, x[r][v].z & 0x7fff7fffu);
        m = __vmaxu2(m, x[r][v].w & 0x7fff7fffu);
      }
      m = max(m & 0xffffu, m >> 16);
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = row_exponent(m);
      const float f = __uint_as_float((uint32_t)e << 23);
      const float sl = p.scale_log2 * exp2f((float)(127 - e));
      if (r == 0) sl0 = sl;
      else sl1 = sl;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const uint32_t w[4] = {x[r][v].x, x[r][v].y, x[r][v].z, x[r][v].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          qa[2 * v + (k >> 1)][r + 2 * (k & 1)] =
              pack_f16x2(bf16lo(w[k]) * f, bf16hi(w[k]) * f);
      }
    }
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int nt = 0; nt < 16; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][j] = 0.f;
  };

  // The unit's state of every warp into the slot, then its rows as outputs
  // (a unit wholly in this CTA's range) or as this CTA's partial of it, by
  // all consumers: M = max m_w, L = sum l_w 2^(m_w - M), row = sum_w
  // 2^(m_w - M) o_w / L.
  auto finish_unit = [&](int b, int h) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    float *wm = slot;                    // [warp][16]
    float *wl = wm + kWarps * kFewRows;  // [warp][16]
    float *wo = wl + kWarps * kFewRows;  // [warp][16][D]
    named_sync(kConsBar, kConsumers);    // the slot is free
    if (qc == 0) {
      wm[warp * 16 + qr] = m0;
      wm[warp * 16 + qr + 8] = m1;
      wl[warp * 16 + qr] = l0;
      wl[warp * 16 + qr + 8] = l1;
    }
    // accumulator column n = 2 qc + (j & 1) of tile nt is dim 16 n + nt
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = qr + (j >= 2 ? 8 : 0);
      float *dst = wo + (warp * 16 + row) * kD + 16 * (2 * qc + (j & 1));
#pragma unroll
      for (int v = 0; v < 4; ++v)
        reinterpret_cast<float4 *>(dst)[v] =
            make_float4(o[4 * v][j], o[4 * v + 1][j], o[4 * v + 2][j],
                        o[4 * v + 3][j]);
    }
    named_sync(kConsBar, kConsumers);
    const int ustart = wp.pre[b] + h * wp.nch[b];
    const int uend = ustart + wp.nch[b];
    const bool whole = ustart >= lo && uend <= hi;
    const long wslot = c * 2 + partial_side(ustart, lo);
    const int rows = un * G;
    for (int jg = warp; jg < HP * rows; jg += kWarps) {
      const int j = jg / rows, g = jg - j * rows, w0 = j * C::WPH;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < C::WPH; ++w) M = fmaxf(M, wm[(w0 + w) * 16 + g]);
      float L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < C::WPH; ++w) {
        const float mw = wm[(w0 + w) * 16 + g];
        const float cw = mw == -INFINITY ? 0.f : ex2(mw - M);
        L = fmaf(wl[(w0 + w) * 16 + g], cw, L);
        const float4 v =
            reinterpret_cast<const float4 *>(wo + ((w0 + w) * 16 + g) *
                                                      kD)[lane];
        acc.x = fmaf(cw, v.x, acc.x);
        acc.y = fmaf(cw, v.y, acc.y);
        acc.z = fmaf(cw, v.z, acc.z);
        acc.w = fmaf(cw, v.w, acc.w);
      }
      // a NaN in a row's scores stays one: its L is NaN
      const float f = L == 0.f ? 0.f : 1.f / L;
      acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
      const float lse = L == 0.f ? -INFINITY
                                 : (M + log2f(L)) * 0.69314718055994531f;
      if (whole) {
        const long at = (urow + g / G) * p.n_h + (long)(h * HP + j) * G +
                        g % G;
        uint2 packed;
        packed.x = pack_bf16x2(acc.x, acc.y);
        packed.y = pack_bf16x2(acc.z, acc.w);
        reinterpret_cast<uint2 *>(p.out + at * kD)[lane] = packed;
        if (lane == 0 && p.lse) p.lse[at] = lse;
      } else {
        const long at = wslot * C::GU + j * kFewRows + g;
        reinterpret_cast<float4 *>(p.ws_o + at * kD)[lane] = acc;
        if (lane == 0) p.ws_lse[at] = lse;
      }
    }
  };

  ChunkCursor cc = cursor_at(wp, p.batch, lo);
  int s = 0, ph = 0;
  for (int i = 0; i < n; ++i) {
    if (cc.b != cur_b || cc.h != cur_h) {
      if (cur_b >= 0) finish_unit(cur_b, cur_h);
      cur_b = cc.b;
      cur_h = cc.h;
      start_unit(cur_b, cur_h);
    }
    ok = ok && !s_abort && mbar_wait(&full[s], ph);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok && lane == 0) {
      if (!s_abort) report(p.err, DEVERR_TIMEOUT);
      s_abort = 1;
    }
    const int T = wp.len[cc.b];
    const int ctok = seq_first(p, cc.b, T, CH) + cc.k * CH;
    if (ok) {
      const uint8_t *kb = sk + s * C::STAGE + hj * CH * kRow;
      const uint8_t *vb = sv + s * C::STAGE + hj * CH * kRow;
      float sc[C::NSUB][2][4];
#pragma unroll
      for (int u = 0; u < C::NSUB; ++u)
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[u][t2][j] = 0.f;
          const uint8_t *row = kb + (wt0 + 16 * u + 8 * t2 + qr) * kRow;
          const uint2 c0 = *reinterpret_cast<const uint2 *>(row + 16 * qc);
          const uint2 c1 = *reinterpret_cast<const uint2 *>(row + 16 * qc + 8);
          const uint32_t sp = e4m3x2_to_f16x2(
              *reinterpret_cast<const uint16_t *>(row + 64 + 2 * qc));
          const uint32_t s0 = prmt(sp, 0, 0x1010), s1 = prmt(sp, 0, 0x3232);
          const uint32_t w[4] = {c0.x, c0.y, c1.x, c1.y};
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const uint32_t sh = k4 < 2 ? s0 : s1;
            uint32_t x[4];
            e2m1x8_to_f16(w[k4], x);
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2)
              mma_f16(sc[u][t2], qa[2 * k4 + h2], mul_f16x2(x[2 * h2], sh),
                      mul_f16x2(x[2 * h2 + 1], sh));
          }
        }
      // ---- online softmax over the warp's tokens, rows qr and qr + 8 ----
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int u = 0; u < C::NSUB; ++u)
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int pos = ctok + wt0 + 16 * u + 8 * t2 + 2 * qc + j;
            sc[u][t2][j] = pos >= lo0 && pos < hi0 ? sc[u][t2][j] * sl0
                                                   : -INFINITY;
            sc[u][t2][2 + j] = pos >= lo1 && pos < hi1
                                   ? sc[u][t2][2 + j] * sl1
                                   : -INFINITY;
          }
          mx0 = fmaxf(mx0, fmaxf(sc[u][t2][0], sc[u][t2][1]));
          mx1 = fmaxf(mx1, fmaxf(sc[u][t2][2], sc[u][t2][3]));
        }
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
      const float u0 = n0 == -INFINITY ? 0.f : n0;
      const float u1 = n1 == -INFINITY ? 0.f : n1;
      const float f0 = ex2(m0 - u0), f1 = ex2(m1 - u1);
      m0 = n0;
      m1 = n1;
      uint32_t pa[C::NSUB][4];
      float ls0 = 0.f, ls1 = 0.f;
#pragma unroll
      for (int u = 0; u < C::NSUB; ++u)
#pragma unroll
        for (int t2 = 0; t2 < 2; ++t2) {
          const float a0 = ex2(sc[u][t2][0] - u0);
          const float a1 = ex2(sc[u][t2][1] - u0);
          const float b0 = ex2(sc[u][t2][2] - u1);
          const float b1 = ex2(sc[u][t2][3] - u1);
          ls0 += a0 + a1;
          ls1 += b0 + b1;
          pa[u][2 * t2] = pack_f16x2(a0, a1);
          pa[u][2 * t2 + 1] = pack_f16x2(b0, b1);
        }
      l0 = l0 * f0 + ls0;
      l1 = l1 * f1 + ls1;
#pragma unroll
      for (int nt = 0; nt < 16; ++nt) {
        o[nt][0] *= f0;
        o[nt][1] *= f0;
        o[nt][2] *= f1;
        o[nt][3] *= f1;
      }
      // ---- O += P V ----
      const bool edge = ctok + wt0 < ulo || ctok + wt0 + C::TPW > T;
#pragma unroll
      for (int u = 0; u < C::NSUB; ++u) {
        uint32_t e[2][2], d[2][2];  // [token pair][word]: even, odd dims
        uint32_t sp[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int tk = wt0 + 16 * u + 8 * t + 2 * qc;
          const uint8_t *row = vb + tk * kRow;
          const uint2 x = *reinterpret_cast<const uint2 *>(row + 8 * qr);
          const uint2 y =
              *reinterpret_cast<const uint2 *>(row + kRow + 8 * qr);
          uint32_t a = row[64 + qr], b = row[kRow + 64 + qr];
          if (edge) {
            // rows outside the unit's positions were not copied: their
            // scales are taken as 0, so that 0 times them stays 0
            const int pos = ctok + tk;
            if (pos < ulo || pos >= T) a = 0;
            if (pos + 1 < ulo || pos + 1 >= T) b = 0;
          }
          sp[t] = e4m3x2_to_f16x2((uint16_t)(a | (b << 8)));
          e[t][0] = (x.x & 0x0f0f0f0fu) | ((y.x & 0x0f0f0f0fu) << 4);
          e[t][1] = (x.y & 0x0f0f0f0fu) | ((y.y & 0x0f0f0f0fu) << 4);
          d[t][0] = ((x.x >> 4) & 0x0f0f0f0fu) | (y.x & 0xf0f0f0f0u);
          d[t][1] = ((x.y >> 4) & 0x0f0f0f0fu) | (y.y & 0xf0f0f0f0u);
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t x[2][4], y[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            e2m1x8_to_f16(e[t][w], x[t]);
            e2m1x8_to_f16(d[t][w], y[t]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma_f16(o[8 * w + 2 * i], pa[u], mul_f16x2(x[0][i], sp[0]),
                    mul_f16x2(x[1][i], sp[1]));
            mma_f16(o[8 * w + 2 * i + 1], pa[u], mul_f16x2(y[0][i], sp[0]),
                    mul_f16x2(y[1][i], sp[1]));
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    cursor_next(wp, p.batch, n_units, cc);
    if (++s == C::NS) s = 0, ph ^= 1;
  }
  if (cur_b >= 0) finish_unit(cur_b, cur_h);

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
// share (as merge_dense_kernel, with a unit's rows spread over sequences'
// rows): four lanes per float4 of outputs, two rows a CTA.
constexpr int kRowMergeThreads = 256;

template <int NB>
__global__ void __launch_bounds__(kRowMergeThreads)
    merge_few_kernel(const __grid_constant__ ExtendParams p, int n_units,
                     int hp, int chunk) {
  __shared__ WorkPartitionT<NB> wp;
  __shared__ int s_len_err;
  pdl_trigger();
  // the lengths and row lists are read before the launch before completes:
  // it does not write them, and it lets this one start only after its own
  // predecessor has completed
  build_partition(wp, p, &s_len_err, chunk, n_units);
  pdl_wait();
  const int total = wp.total;
  if (total == 0) return;
  const int P = min(p.n_splits, total);
  const int G = p.n_h / p.n_kv;
  const int u = blockIdx.x;
  const int b = u / n_units, h = u - b * n_units;
  if (wp.nch[b] == 0) return;
  const int ustart = wp.pre[b] + h * wp.nch[b];
  const int c_first = cta_of(ustart, total, P);
  const int parts = cta_of(ustart + wp.nch[b] - 1, total, P) - c_first + 1;
  if (parts == 1) return;
  const int rows = seq_rows(p, b) * G;
  const int gu = hp * kFewRows;
  const long row0 = p.row_start ? p.row_start[b] : b;
  auto slot = [&](int i) { return (long)(c_first + i) * 2 + (i == 0 ? 1 : 0); };
  const int x = threadIdx.x & 127;  // 32 float4 x 4 lanes
  for (int jg = blockIdx.y * 2 + (threadIdx.x >> 7); jg < hp * rows;
       jg += gridDim.y * 2) {
    const int j = jg / rows, g = jg - j * rows;
    const int sl = j * kFewRows + g, e4 = x >> 2;
    float M, W;
    float4 acc;
    quad_merge<4>(p.ws_lse, p.ws_o, gu, kD, sl, sl * (kD / 4) + e4, parts,
                  slot, M, W, acc);
    if ((x & 3) == 0) {
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
}

template <int HP, int CH>
cudaError_t launch_few_t(const ExtendParams &p, cudaStream_t s) {
  using C = FCfg<HP, CH>;
  auto kern = extend_few_kernel<HP, CH>;
  static bool done[64] = {};
  cudaError_t e = set_smem_once(kern, C::SMEM, done);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(p.n_splits), dim3(kThreads), C::SMEM, s, 1, p);
  if (e != cudaSuccess || p.whole_units || p.n_splits <= 1) return e;
  const int n_units = p.n_kv / HP;
  const int rows = HP * std::min(kFewRows, p.max_rows * (p.n_h / p.n_kv));
  const dim3 grid(p.batch * n_units, (rows + 1) / 2);
  if (p.batch <= kMergeSmallBatch)
    return launch_pdl(merge_few_kernel<kMergeSmallBatch>, grid,
                      dim3(kRowMergeThreads), 0, s, 1, p, n_units, HP, CH);
  return launch_pdl(merge_few_kernel<kMaxDecodeBatch>, grid,
                    dim3(kRowMergeThreads), 0, s, 1, p, n_units, HP, CH);
}

}  // namespace

// Two heads a unit where a block holds a 64-position chunk of both side by
// side (one 9 KB copy instead of two).
int extend_few_heads(int n_kv, int block_size) {
  return block_size == 64 && n_kv % 2 == 0 ? 2 : 1;
}
// One head a unit: 128 positions give each of the eight warps its 16.
int extend_few_chunk(int hp) { return hp == 2 ? 64 : 128; }

cudaError_t launch_extend_few(const ExtendParams &p, cudaStream_t s) {
  if (p.batch > kMaxDecodeBatch) return cudaErrorNotSupported;
  return p.hp == 2 ? launch_few_t<2, 64>(p, s) : launch_few_t<1, 128>(p, s);
}

}  // namespace kvd
