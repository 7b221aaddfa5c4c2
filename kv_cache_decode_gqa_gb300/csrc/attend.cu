// Attention of several rows a sequence that is not causal (kvd_gqa_tree,
// kvd_gqa_cross): the plan of a call, the launches, and the merge of the units
// that CTAs share.
#include "attend_tc.cuh"

namespace kvd {
namespace {

// Log-sum-exp merge of the units that several CTAs of the launch before share:
// CTA (c - 1, y) looks whether that launch's CTA c is the first to begin inside
// a unit, and then merges the unit's parts of every gridDim.y-th group of
// pairs, a lane a float4 of an output row and up to 8 parts' loads in flight.
// The work is scanned and the unit found while the other launch's last CTAs
// still run (it lets this one start only after its own predecessor has
// completed).
constexpr int kAttendMergeThreads = 256;

template <int D, int NB>
__global__ void __launch_bounds__(kAttendMergeThreads)
    attend_merge_kernel(const __grid_constant__ AttendParams p) {
  __shared__ long scratch[33], s_start;
  __shared__ int s_seq;
  __shared__ Seq s_q;
  pdl_trigger();
  const int G = p.n_h / p.n_kv, tid = threadIdx.x;
  constexpr int SPT = (NB + kAttendMergeThreads - 1) / kAttendMergeThreads;
  Seq sq[SPT];
  long before, total;
  int end;
  scan_work(p, G, scratch, sq, before, total, end);
  // (every CTA waits, also one that has nothing to merge: what follows this
  // launch on the stream waits for this one only)
  const int P = (int)min((long)p.n_splits, total), c = blockIdx.x + 1;
  if (c >= P) {
    pdl_wait();
    return;
  }
  const long x = share_lo(c, total, P);
  const int per = (p.batch + kAttendMergeThreads - 1) / kAttendMergeThreads;
#pragma unroll
  for (int j = 0; j < SPT; ++j) {
    if (j >= per || tid * per + j >= p.batch) continue;
    const long n = seq_chunks(p, sq[j]);
    if (x >= before && x < before + n) {
      s_seq = tid * per + j;
      s_start = before;
      s_q = sq[j];
    }
    before += n;
  }
  __syncthreads();
  const Seq q = s_q;
  const int len = unit_len(p, q);
  const int unit = (int)div_u(x - s_start, len);
  const long u = s_start + (long)unit * len;  // its first chunk
  // begun by CTA c - 1 and not over when CTA c begins?
  const bool cut = u < x && share_lo(c - 1, total, P) <= u && x - u < q.nch;
  pdl_wait();
  if (!cut) return;
  const int parts = share_of(u + q.nch - 1, total, P) - (c - 1) + 1;
  const int h = unit / q.blocks, f0 = (unit - h * q.blocks) * kUnit;
  const int np = min(q.n * G - f0, kUnit);
  constexpr int LANES = D / 4, ROWS = kAttendMergeThreads / LANES;
  const int e4 = tid % LANES;
  for (int ri = blockIdx.y * ROWS + tid / LANES; ri < np;
       ri += gridDim.y * ROWS) {
    float M, W;
    float4 acc;
    quad_merge<1>(p.ws_lse, p.ws_o, p.block_rows, D, ri, ri * LANES + e4,
                  parts,
                  [&](int i) { return (long)(c - 1 + i) * 2 + (i == 0); }, M, W,
                  acc);
    const float iw = W == 0.f ? 0.f : 1.f / W;
    const int f = f0 + ri;
    const long at = ((long)q.r0 + f / G) * p.n_h + (long)h * G + f % G;
    uint2 packed;
    packed.x = pack_bf16x2(acc.x * iw, acc.y * iw);
    packed.y = pack_bf16x2(acc.z * iw, acc.w * iw);
    reinterpret_cast<uint2 *>(p.out + at * D)[e4] = packed;
    if (e4 == 0 && p.lse) p.lse[at] = W == 0.f ? -INFINITY : M + logf(W);
  }
}

template <int D>
cudaError_t launch_merge(const AttendParams &p, cudaStream_t s) {
  // a row or two a warp
  const int rows = 2 * kAttendMergeThreads / (D / 4);
  const dim3 grid(p.n_splits - 1, (p.block_rows + rows - 1) / rows);
  return launch_pdl(p.batch <= kAttendMergeThreads
                        ? attend_merge_kernel<D, kAttendMergeThreads>
                        : attend_merge_kernel<D, kMaxDecodeBatch>,
                    grid, dim3(kAttendMergeThreads), 0, s, 1, p);
}

// Two tensors of a bf16 cache (or one, twice) as [which][column half][row][64
// columns], in swizzled boxes of `box` rows (of all columns where box is 64) of
// one of them.
bool cache_map(CUtensorMap *map, const AttendParams &p, const uint8_t *lo,
               const uint8_t *hi, int box) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t d = p.dk;
  const cuuint64_t dims[4] = {
      64, (cuuint64_t)p.num_blocks * p.n_kv * p.block_size, d / 64,
      lo == hi ? 1u : 2u};
  const cuuint64_t strides[3] = {2 * d, 128,
                                 lo == hi ? 16 : (cuuint64_t)(hi - lo)};
  const cuuint32_t boxes[4] = {64, (cuuint32_t)box,
                               (cuuint32_t)(box == 64 ? d / 64 : 1), 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<uint8_t *>(lo), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

constexpr long kMergeChunks = 4, kMinChunks = 4;

AttendPlan attend_plan(int n_kv, int g, int d, int batch, int rows,
                       int max_rows, int max_seq_len, int ctas) {
  AttendPlan pl;
  pl.pairs = (int)std::min((long)max_rows * g, (long)kUnit);
  const long units =
      (long)n_kv * (((long)rows * g + (long)std::min(batch, rows) * (kUnit - 1)) /
                    kUnit);
  const long each = ((long)max_seq_len + kN - 1) / kN;
  const long chunks = units * each;
  // Not cut where a CTA a unit then takes no more than kMergeChunks chunks longer
  // than equal shares would: the merge launch, which finds no room beside CTAs of
  // this one, costs more. (Trees of 16 nodes of 8 heads a kv head, bf16, whole
  // units against shares, us in a graph: 8 units of 3, 5 and 8 chunks 10.3 / 11.5,
  // 11.9 / 21.8, 14.1 / 17.4; 64 units of 5, 8 and 14 chunks 12.6 / 28.4, 15.0 /
  // 31.8, 19.5 / 31.6; 128 units of 18 and 32 chunks 55.2 / 55.5, 73.8 / 73.9; 8
  // units of 32 chunks 42 / 21. fp8 alike.)
  if (units <= ctas && each <= chunks / ctas + kMergeChunks) {
    pl.whole_units = 1;
    pl.ctas = (int)std::max(1L, units);
    return pl;
  }
  // A CTA takes kMinChunks at least: its partial result of a unit of 128 pairs
  // has the bytes of a chunk. (16 nodes of 8 heads each over 4,000 positions,
  // us: 8 CTAs 42, 32 23.3, 64 20.6, 96 23.0, 152 26.8.)
  pl.ctas = (int)std::max(
      1L, std::min((long)ctas, std::max(units, chunks / kMinChunks)));
  // A change of units (its queries, outputs, the filling of the pipeline) counts
  // as kUnitGap chunks where shares are long. (Gaps of 0, 2, 4, 8, 14 chunks, us:
  // fp8 trees 116, 107, 102, 102, 104; 2,003 rows of six ragged sequences 137,
  // 113, 101, 101, 105.)
  if (chunks >= 8L * pl.ctas) pl.gap = kUnitGap;
  if (pl.ctas > 1) {
    const size_t slots = (size_t)pl.ctas * 2 * pl.pairs;
    pl.ws_o_bytes = (slots * d * 4 + 255) / 256 * 256;
    pl.ws_bytes = pl.ws_o_bytes + (slots * 4 + 255) / 256 * 256;
  }
  return pl;
}

cudaError_t launch_attend(const AttendParams &p, cudaStream_t s) {
  TcParams tp{};
  tp.p = p;
  cudaError_t e;
  if (p.dtype == DT_BF16) {
    // boxes of rows that lie within a block and within half a chunk
    tp.box = std::min(64, p.block_size & -p.block_size);
    const uint8_t *lo = std::min(p.k, p.v), *hi = std::max(p.k, p.v);
    tp.far = (hi - lo) >> 40 != 0;
    if (!tp.far) {
      // (one map: half the encoding, and K and V share its fetch)
      if (!cache_map(&tp.map[0], p, lo, hi, tp.box))
        return cudaErrorNotSupported;
      tp.which[0] = p.v < p.k;
      tp.which[1] = p.k < p.v;
    } else if (!cache_map(&tp.map[0], p, p.k, p.k, tp.box) ||
               !cache_map(&tp.map[1], p, p.v, p.v, tp.box)) {
      return cudaErrorNotSupported;
    }
    e = p.dk == 128 ? launch_attend_t<DT_BF16, 128, 2>(tp, s)
                    : launch_attend_t<DT_BF16, 64, 2>(tp, s);
  } else {
    e = launch_attend_widen(tp, p.block_rows <= kM, s);
  }
  if (e != cudaSuccess || p.n_splits <= 1 || p.whole_units) return e;
  return p.dk == 128 ? launch_merge<128>(p, s) : launch_merge<64>(p, s);
}

}  // namespace kvd
