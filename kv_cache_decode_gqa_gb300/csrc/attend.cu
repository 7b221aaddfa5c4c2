// Attention of several rows a sequence that is not causal (kvd_gqa_tree,
// kvd_gqa_cross): the launches, and the merge of the units that CTAs share.
#include "attend_tc.cuh"

namespace kvd {
namespace {

// Log-sum-exp merge of the units that several CTAs of the launch before share:
// a lane a float4 of an output row, up to 8 parts' loads in flight. A CTA is
// small enough to sit beside one of that launch, so that the work is scanned
// and the rows' parts are found while it still runs (it lets this one start
// only after its own predecessor has completed).
constexpr int kAttendMergeThreads = 256;

template <int D, int NB>
__global__ void __launch_bounds__(kAttendMergeThreads)
    attend_merge_kernel(const __grid_constant__ AttendParams p) {
  __shared__ long scratch[33], pre[NB];
  pdl_trigger();
  const int G = p.n_h / p.n_kv, tid = threadIdx.x;
  constexpr int SPT = (NB + kAttendMergeThreads - 1) / kAttendMergeThreads;
  Seq sq[SPT];
  long before, total;
  int end;
  scan_work(p, G, scratch, sq, before, total, end);
  const int per = (p.batch + kAttendMergeThreads - 1) / kAttendMergeThreads;
#pragma unroll
  for (int j = 0; j < SPT; ++j) {
    if (j >= per || tid * per + j >= p.batch) continue;
    pre[tid * per + j] = before;
    before += seq_chunks(p, sq[j]);
  }
  __syncthreads();
  const int P = (int)min((long)p.n_splits, total);
  constexpr int LANES = D / 4;  // of a row
  const long at = (long)blockIdx.x * (kAttendMergeThreads / LANES) +
                  tid / LANES;
  const int e4 = tid % LANES;
  int parts = 0, first = 0, ri = 0;
  if (at < (long)p.rows * p.n_h) {
    const int row = (int)(at / p.n_h), head = (int)(at - (long)row * p.n_h);
    int b = 0;
    Seq q{};
    for (; b < end; ++b) {
      const int r0 = p.row_start ? p.row_start[b] : b;
      const int r1 = p.row_start ? p.row_start[b + 1] : b + 1;
      if (row >= r0 && row < r1) {
        q = seq_at(p, b, G);
        break;
      }
    }
    if (q.n > 0 && q.nch > 0) {
      const int f = (row - q.r0) * G + head % G, m = f / kUnit;
      ri = f - m * kUnit;
      const long u =
          pre[b] + ((long)(head / G) * q.blocks + m) * q.nch;
      first = share_of(u, total, P);
      parts = share_of(u + q.nch - 1, total, P) - first + 1;
    }
  }
  pdl_wait();
  if (parts <= 1) return;  // written whole, or no sequence's row
  float M, W;
  float4 acc;
  quad_merge<1>(p.ws_lse, p.ws_o, p.block_rows, D, ri, ri * LANES + e4, parts,
                [&](int i) { return (long)(first + i) * 2 + (i == 0); }, M, W,
                acc);
  const float iw = W == 0.f ? 0.f : 1.f / W;
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * iw, acc.y * iw);
  packed.y = pack_bf16x2(acc.z * iw, acc.w * iw);
  reinterpret_cast<uint2 *>(p.out + at * D)[e4] = packed;
  if (e4 == 0 && p.lse) p.lse[at] = W == 0.f ? -INFINITY : M + logf(W);
}

template <int D>
cudaError_t launch_merge(const AttendParams &p, cudaStream_t s) {
  const long rows = (long)p.rows * p.n_h;
  const long per = kAttendMergeThreads / (D / 4);
  const dim3 grid((unsigned)((rows + per - 1) / per));
  return launch_pdl(p.batch <= kMergeSmallBatch
                        ? attend_merge_kernel<D, kMergeSmallBatch>
                        : attend_merge_kernel<D, kMaxDecodeBatch>,
                    grid, dim3(kAttendMergeThreads), 0, s, 1, p);
}

// A bf16 cache as [column half][row][64 columns], in swizzled boxes of `box`
// rows (of all columns where box is 64).
bool cache_map(CUtensorMap *map, const uint8_t *data, const AttendParams &p,
               int box) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t d = p.dk;
  const cuuint64_t dims[3] = {
      64, (cuuint64_t)p.num_blocks * p.n_kv * p.block_size, d / 64};
  const cuuint64_t strides[2] = {2 * d, 128};
  const cuuint32_t boxes[3] = {64, (cuuint32_t)box,
                               (cuuint32_t)(box == 64 ? d / 64 : 1)};
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                const_cast<uint8_t *>(data), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

AttendPlan attend_plan(int n_kv, int g, int d, int batch, int rows,
                       int max_rows, int max_seq_len, int ctas) {
  AttendPlan pl;
  pl.pairs = (int)std::min((long)max_rows * g, (long)kUnit);
  const long units =
      (long)n_kv * (((long)rows * g + (long)std::min(batch, rows) * (kUnit - 1)) /
                    kUnit);
  const long chunks = units * (((long)max_seq_len + kN - 1) / kN);
  pl.ctas = (int)std::max(1L, std::min((long)ctas, chunks));
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
    if (!cache_map(&tp.tmk, p.k, p, tp.box) ||
        !cache_map(&tp.tmv, p.v, p, tp.box))
      return cudaErrorNotSupported;
    e = p.dk == 128 ? launch_attend_t<DT_BF16, 128, 2>(tp, s)
                    : launch_attend_t<DT_BF16, 64, 2>(tp, s);
  } else {
    e = launch_attend_widen(tp, p.block_rows <= kM, s);
  }
  if (e != cudaSuccess || p.n_splits <= 1) return e;
  return p.dk == 128 ? launch_merge<128>(p, s) : launch_merge<64>(p, s);
}

}  // namespace kvd
