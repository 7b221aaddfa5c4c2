// Ragged rows in and out of the paged cache: rotary positions (kvd_rope),
// the write of new rows with the rotation fused into it (kvd_kv_write) and
// the read of cached rows as bf16 (kvd_kv_read).
//
// Rotation: pair i of a row turns by positions[axis_i][row] * f_i. f_i comes
// as a 64-bit fixed-point fraction of a turn, so position * turns wraps
// modulo 2^64 exactly where the angle wraps modulo a turn: the top 32 bits
// of the wrapped product are the angle (to 2^-32 of a turn, whatever the
// position), and sincospi takes it without a range reduction. A CTA takes a
// few consecutive rows, forms each row's d_rot / 2 cosines and sines once in
// shared memory and applies them to every head, 16 bytes a thread and load.
//
// All three are bound by HBM: a row is read once and written once. The
// sine/cosine work (64 pairs a row, about 40 instructions each) is spread
// over the CTA's threads and is 4% of a row's time at 72 heads. Measured:
// 16,384 rows of 72 heads turned in 102 us (604 MB, 5.9 TB/s; the same in
// CTAs of 128 or 512 threads or six an SM: slower, up to 131 us); 12,007 rows
// of 64 heads turned and of 8 + 8 heads turned and stored, in E4M3 in 90 us
// (467 MB, 5.2 TB/s), in 4 bits in 86 us; 110,003 rows of 8 + 8 heads read
// from 4 bits in 96 us (577 MB, 6.0 TB/s), from E4M3 in 133 us (5.1 TB/s), from
// bf16 in 143 us (6.3 TB/s). The loads of a thread's next 16 bytes are issued
// before it finishes these (106 us without, for the first figure).
//
// Write: with a rotation the turned keys pass through shared memory as bf16
// (the rounding kvd_rope would make), then every row is encoded exactly as
// kv_append encodes it. The MXFP4 encoder divides by one reciprocal per
// 16-channel group instead of 16 exact divisions (mxfp4_group). Rows without a
// rotation do not reach the copy rate: 30,011 rows of 8 + 8 heads take 41 us in
// 4 bits (157 MB, 3.8 TB/s), 53 in E4M3 and 56 in bf16. In 4 bits the kernel
// issues 260 instructions a group on 64% of its slots (addresses are formed
// anew for each group), and waits longest for the group's own loads, which
// nothing issues ahead.
#include <algorithm>

#include "prompt_common.cuh"

namespace kvd {
namespace {

constexpr int kThreads = 256;

// One 16-channel group of bf16 values (8 words) as E2M1 codes and an E4M3
// scale, the same bytes as store_mxfp4_group. There each code is E2M1(q),
// q = x / s correctly rounded, i.e. decided by comparing q with the
// midpoints m of the grid. Here fma(x, 1 / s, M) - M, M = 1.5 * 2^12, gives q
// rounded to a multiple of 2^-11. x has 8 significand bits and m s at most 7,
// so x / s is either m or at least m / 256 >= 2^-10 away from it: a tie comes
// out as m (a multiple of 1/4) although 1 / s is rounded, and no other value
// passes a midpoint. Values of 8 and more, where M no longer rounds like
// that, and infinities saturate either way. The hardware conversion then
// rounds ties to even and saturates as e2m1_code does. Groups that hold a NaN
// take the plain path.
__device__ __forceinline__ void mxfp4_group(uint8_t *codes, uint8_t *scale,
                                            const uint16_t *src) {
  const uint4 u0 = *reinterpret_cast<const uint4 *>(src);
  const uint4 u1 = *reinterpret_cast<const uint4 *>(src + 8);
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  // |x| of bf16 values orders as their low 15 bits do
  uint32_t m2 = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, w[j] & 0x7fff7fffu);
  const uint32_t mb = max(m2 & 0xffffu, m2 >> 16);
  if (mb > 0x7f80u) {  // a NaN
    store_mxfp4_group(codes, scale, src);
    return;
  }
  const float amax = __uint_as_float(mb << 16);
  const uint32_t sc = e4m3x2_from_f32(__fdiv_rn(amax, 6.0f), 0.f) & 0xffu;
  const float s = f16lo(e4m3x2_to_f16x2((uint16_t)sc));
  uint32_t packed[2] = {0u, 0u};
  if (s > 0.f) {
    const float r = __fdiv_rn(1.0f, s);
    constexpr float kMagic = 6144.0f;  // 1.5 * 2^12: ulp 2^-11
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x0 = bf16lo(w[j]), x1 = bf16hi(w[j]);
      // the sign of a value that rounds to 0 is kept (as e2m1_code keeps it)
      const float q0 = copysignf(fmaf(x0, r, kMagic) - kMagic, x0);
      const float q1 = copysignf(fmaf(x1, r, kMagic) - kMagic, x1);
      uint32_t b;
      asm("{\n\t.reg .b8 t;\n\t"
          "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
          "cvt.u32.u8 %0, t;\n\t}"
          : "=r"(b)
          : "f"(q0), "f"(q1));
      packed[j >> 2] |= (b & 0xffu) << (8 * (j & 3));
    }
  }
  *reinterpret_cast<uint2 *>(codes) = make_uint2(packed[0], packed[1]);
  *scale = (uint8_t)sc;
}

// cos and sin of position * turns (see above).
__device__ __forceinline__ float2 turn(uint64_t turns, int pos, bool inverse) {
  const uint32_t frac =
      (uint32_t)((turns * (uint64_t)(int64_t)pos) >> 32);  // modulo 2^64
  // in half turns, [-1, 1)
  const float h = (float)(int32_t)frac * 0x1p-31f;
  float s, c;
  sincospif(h, &s, &c);
  return make_float2(c, inverse ? -s : s);
}

// Eight E2M1 codes times their group's scale as bf16, exactly (6 significand
// bits), through fp32. (Packed bf16 multiplications of the shifted f16 codes
// take fewer instructions and ran 10% slower.)
__device__ __forceinline__ void mxfp4_to_bf16(uint32_t codes, float scale,
                                              uint32_t (&o)[4]) {
  uint32_t h[4];
  e2m1x8_to_f16(codes, h);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = pack_bf16x2(f16lo(h[j]) * scale, f16hi(h[j]) * scale);
}

// The sequence of ragged row r, or -1 for padding.
__device__ __forceinline__ int seq_of_row(const int32_t *row_start, int batch,
                                          int r) {
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (row_start[mid] <= r)
      lo = mid;
    else
      hi = mid - 1;
  }
  return r >= row_start[lo] && r < row_start[lo + 1] ? lo : -1;
}

constexpr long kPadding = -1;   // a row that no sequence owns
constexpr long kBadPos = -2;    // a position outside the block table
constexpr long kBadBlock = -3;  // a block id out of range

// First element row of ragged row r's slot (head 0), or one of the above. A
// sequence that starts below 0 or ends past the rows owns none.
__device__ __forceinline__ long slot_of_row(const RowsParams &p, int r) {
  const int b = seq_of_row(p.row_start, p.batch, r);
  if (b < 0) return kPadding;
  const int first = p.row_start[b];
  if (first < 0 || p.row_start[b + 1] > p.rows) return kPadding;
  const long pos = (long)p.start[b] + (r - first);
  if (pos < 0 || pos >= (long)p.max_blocks * p.block_size) return kBadPos;
  const int blk =
      p.block_table[(long)b * p.max_blocks + (int)(pos / p.block_size)];
  if (blk < 0 || blk >= p.num_blocks) return kBadBlock;
  return (long)blk * p.n_kv * p.block_size + (int)(pos % p.block_size);
}

// Row lists up to this long are gone through by every CTA (warps 1 to 7, in up
// to 10 rounds of loads, beside the first warp's bisections: nothing on the
// clock), longer ones a share by each: 65,535 entries would cost a CTA more
// than its rows.
constexpr int kListChecked = 2048;

// Whether this thread finds that the list descends, which makes bisections
// meaningless: the call then does nothing. (A second search, for what lies
// before the descent, costs good lists too: 40 registers in read_kernel instead
// of 32, 96 to 106 us; as another turn of one loop, 112 to 113.5 us for the
// turned fp8 write.) Bad entries are flagged once, or by the CTA whose share
// they are in. The caller's __syncthreads_or shares the answer and the slots.
__device__ __forceinline__ bool list_descends(const RowsParams &p) {
  const bool all = p.batch <= kListChecked;
  const bool flag = !all || (blockIdx.x == 0 && blockIdx.y == 0);
  bool broken = false;
  int b = (int)threadIdx.x - 32, step = kThreads - 32;
  if (b < 0) return false;
  if (!all) {  // (65,536 CTAs are enough for every list)
    b = blockIdx.y == 0 && blockIdx.x < 65536u ? b + (int)blockIdx.x * step
                                               : p.batch;
    step *= (int)min(gridDim.x, 65536u);
  }
#pragma unroll 1
  for (; b < p.batch; b += step) {
    const int x = p.row_start[b], y = p.row_start[b + 1];
    broken |= y < x;
    if (flag && x != y && (y < x || x < 0 || y > p.rows))
      report(p.err, DEVERR_LEN);
  }
  return broken && all;
}

__device__ __forceinline__ void report_slot(const RowsParams &p, long slot) {
  if (slot < kPadding)
    report(p.err, slot == kBadPos ? DEVERR_POS : DEVERR_BLOCK);
}

// Threads per row-head: the pieces of one, rounded up to a power of two.
__device__ __forceinline__ int lanes_for(int pieces) {
  int l = 1;
  while (l < pieces && l < kThreads) l <<= 1;
  return l;
}

__device__ __forceinline__ uint32_t rot_lo(uint32_t a, uint32_t b, float2 c0,
                                           float2 c1) {
  return pack_bf16x2(fmaf(bf16lo(a), c0.x, -(bf16lo(b) * c0.y)),
                     fmaf(bf16hi(a), c1.x, -(bf16hi(b) * c1.y)));
}
__device__ __forceinline__ uint32_t rot_hi(uint32_t a, uint32_t b, float2 c0,
                                           float2 c1) {
  return pack_bf16x2(fmaf(bf16lo(b), c0.x, bf16lo(a) * c0.y),
                     fmaf(bf16hi(b), c1.x, bf16hi(a) * c1.y));
}

// One piece of the rotation of a row-head: 16-byte pieces of 8 pairs (half)
// or 4 (adjacent), then of 8 channels that stay. Loading and finishing are
// apart so that the next piece's loads are in flight meanwhile.
struct RotPiece {
  uint16_t *dst;
  const float2 *cs;
  uint4 x, y;
  int c;
};

__device__ __forceinline__ void load_piece(const RopeParams &rp, int nrot,
                                           const uint16_t *src, RotPiece &q) {
  const int c = q.c;
  if (c >= nrot) {  // channels past d_rot
    q.x = *reinterpret_cast<const uint4 *>(src + 2 * rp.half + (c - nrot) * 8);
  } else {
    q.x = *reinterpret_cast<const uint4 *>(src + c * 8);
    if (!rp.adjacent)
      q.y = *reinterpret_cast<const uint4 *>(src + rp.half + c * 8);
  }
}

__device__ __forceinline__ void finish_piece(const RopeParams &rp, int nrot,
                                             const RotPiece &q) {
  const int half = rp.half, c = q.c;
  uint16_t *dst = q.dst;
  const float2 *cs = q.cs;
  if (c >= nrot) {
    *reinterpret_cast<uint4 *>(dst + 2 * half + (c - nrot) * 8) = q.x;
  } else if (rp.adjacent) {
    uint32_t w[4] = {q.x.x, q.x.y, q.x.z, q.x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 t = cs[c * 4 + j];
      const float a = bf16lo(w[j]), b = bf16hi(w[j]);
      w[j] = pack_bf16x2(fmaf(a, t.x, -(b * t.y)), fmaf(b, t.x, a * t.y));
    }
    *reinterpret_cast<uint4 *>(dst + c * 8) =
        make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const uint32_t a[4] = {q.x.x, q.x.y, q.x.z, q.x.w};
    const uint32_t b[4] = {q.y.x, q.y.y, q.y.z, q.y.w};
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 t = *reinterpret_cast<const float4 *>(cs + c * 8 + 2 * j);
      const float2 t0 = make_float2(t.x, t.y), t1 = make_float2(t.z, t.w);
      lo[j] = rot_lo(a[j], b[j], t0, t1);
      hi[j] = rot_hi(a[j], b[j], t0, t1);
    }
    *reinterpret_cast<uint4 *>(dst + c * 8) =
        make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4 *>(dst + half + c * 8) =
        make_uint4(hi[0], hi[1], hi[2], hi[3]);
  }
}

// The same element by element, where no 16-byte access fits: pair c, or
// channel half + c past d_rot.
__device__ __forceinline__ void rotate_pair(const RopeParams &rp,
                                            const uint16_t *src, uint16_t *dst,
                                            const float2 *cs, int c) {
  if (c >= rp.half) {
    const int at = rp.half + c;  // 2 * half + (c - half)
    dst[at] = src[at];
    return;
  }
  const int i = rp.adjacent ? 2 * c : c;
  const int j = rp.adjacent ? 2 * c + 1 : c + rp.half;
  const float a = __uint_as_float((uint32_t)src[i] << 16);
  const float b = __uint_as_float((uint32_t)src[j] << 16);
  const float2 t = cs[c];
  dst[i] = f2bf(fmaf(a, t.x, -(b * t.y)));
  dst[j] = f2bf(fmaf(b, t.x, a * t.y));
}

// WRITE: the cache write (dtype DT), else the rotation alone. A CTA takes
// rows [tile * blockIdx.x, + tile) and the blockIdx.y-th share of the heads.
template <bool VEC, bool WRITE, int DT>
__global__ void __launch_bounds__(kThreads, 5)
    rows_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long s_slot[kMaxRowTile];
  const RopeParams &rp = p.rope;
  const int tid = threadIdx.x;
  const int r0 = (int)blockIdx.x * p.tile;
  const int nr = min(p.tile, p.rows - r0);
  const int ys = gridDim.y, y = blockIdx.y;
  const int qh0 = (int)((long)p.n_h * y / ys);
  const int nq = (int)((long)p.n_h * (y + 1) / ys) - qh0;
  const int kh0 = (int)((long)p.n_kv * y / ys);
  const int nk = (int)((long)p.n_kv * (y + 1) / ys) - kh0;
  float2 *cs = reinterpret_cast<float2 *>(smem);  // [tile][half]
  uint16_t *sk = reinterpret_cast<uint16_t *>(
      smem + (rp.on ? (size_t)p.tile * rp.half * 8 + 15 & ~(size_t)15 : 0));
  pdl_trigger();
  pdl_wait();
  bool broken = false;
  if constexpr (WRITE) {
    if (tid < nr) s_slot[tid] = slot_of_row(p, r0 + tid);
    broken = list_descends(p);
  }
  if (rp.on) {
    for (int i = tid; i < nr * rp.half; i += kThreads) {
      const int r = i / rp.half, pr = i - r * rp.half;
      int ax = rp.axis ? rp.axis[pr] : 0;
      if (ax >= rp.n_axes) {
        report(p.err, DEVERR_INDEX);
        ax = 0;
      }
      const int pos = rp.pos[(long)ax * rp.axis_stride + r0 + r];
      cs[i] = turn(rp.turns[pr], pos, rp.inverse);
    }
  }
  if constexpr (WRITE) {
    if (__syncthreads_or(broken)) return;
    if (tid < nr) report_slot(p, s_slot[tid]);
  } else {
    __syncthreads();
  }
  if (rp.on) {
    const int d = p.d;
    const int nrot = VEC ? (rp.adjacent ? rp.half / 4 : rp.half / 8)
                         : rp.half;
    const int rest = VEC ? (d - 2 * rp.half) / 8 : d - 2 * rp.half;
    const int pieces = nrot + rest;
    const int L = lanes_for(pieces);
    const int heads = nq + nk;
    const int step = kThreads / L;
    int r = 0, h = tid / L;
    // the next row-head of this thread that has a row: source, destination
    auto next = [&](const uint16_t *&src, uint16_t *&dst) {
      for (; heads > 0; h += step) {
        while (h >= heads) h -= heads, ++r;
        if (r >= nr) return false;
        if (WRITE && s_slot[r] == kPadding) continue;
        const long row = r0 + r;
        const bool is_q = h < nq;
        src = is_q ? p.q + row * p.q_rs + (qh0 + h) * p.q_hs
                   : p.k + row * p.k_rs + (kh0 + h - nq) * p.k_hs;
        dst = is_q    ? p.q_out + row * p.qo_rs + (qh0 + h) * p.qo_hs
              : WRITE ? sk + ((long)r * nk + h - nq) * d
                      : p.k_out + row * p.ko_rs + (kh0 + h - nq) * p.ko_hs;
        return true;
      }
      return false;
    };
    const uint16_t *src;
    if constexpr (VEC) {
      // one piece a row-head and thread (at most 256 pieces)
      RotPiece cur, nxt;
      cur.c = nxt.c = tid & (L - 1);
      auto fetch = [&](RotPiece &q) {
        while (next(src, q.dst)) {
          q.cs = cs + r * rp.half;
          h += step;
          // in place the channels past d_rot are already there
          if (q.c < (src == q.dst ? nrot : pieces)) {
            load_piece(rp, nrot, src, q);
            return true;
          }
        }
        return false;
      };
      bool more = fetch(cur);
      while (more) {
        more = fetch(nxt);
        finish_piece(rp, nrot, cur);
        cur = nxt;
      }
    } else {
      uint16_t *dst;
      for (; next(src, dst); h += step) {
        const int end = src == dst ? nrot : pieces;
        for (int c = tid & (L - 1); c < end; c += L)
          rotate_pair(rp, src, dst, cs + r * rp.half, c);
      }
    }
  }
  if constexpr (WRITE) {
    if (rp.on) __syncthreads();
    constexpr int W = DT == DT_MXFP4 ? 16 : 8;
    const int pieces = p.d / W;
    const int L = lanes_for(pieces);
    const int step = kThreads / L;
    const int nt = p.v ? 2 * nk : nk;  // K heads, then V heads
    int r = 0, h = tid / L;
    while (nt > 0) {
      while (h >= nt) h -= nt, ++r;
      if (r >= nr) break;
      const long slot = s_slot[r];
      if (slot >= 0) {
        const bool is_v = h >= nk;
        const int hh = is_v ? h - nk : h;
        const long row = r0 + r;
        const uint16_t *src =
            is_v    ? p.v + row * p.v_rs + (kh0 + hh) * p.v_hs
            : rp.on ? sk + ((long)r * nk + hh) * p.d
                    : p.k + row * p.k_rs + (kh0 + hh) * p.k_hs;
        uint8_t *dst =
            (is_v ? p.v_cache : p.k_cache) +
            (slot + (long)(kh0 + hh) * p.block_size) * row_bytes(p.d, DT);
        float inv = 1.f;
        if (DT == DT_FP8) inv = (is_v ? p.v_inv : p.k_inv)[kh0 + hh];
        for (int c = tid & (L - 1); c < pieces; c += L) {
          if constexpr (DT == DT_MXFP4)
            mxfp4_group(dst + c * 8, dst + p.d / 2 + c, src + c * 16);
          else
            store_new8(dst + c * 8 * (DT == DT_BF16 ? 2 : 1), src + c * 8, DT,
                       inv);
        }
      }
      h += step;
    }
  }
}

// Cached rows as bf16. A row-head is read in pieces of 16 channels (MXFP4)
// or 8; the rows of a head lie side by side in a block, and a CTA takes
// consecutive rows, so its reads cover whole runs of them.
template <int DT>
__global__ void __launch_bounds__(kThreads)
    read_kernel(const __grid_constant__ RowsParams p) {
  __shared__ long s_slot[kMaxRowTile];
  const int tid = threadIdx.x;
  const int r0 = (int)blockIdx.x * p.tile;
  const int nr = min(p.tile, p.rows - r0);
  const int ys = gridDim.y, y = blockIdx.y;
  const int kh0 = (int)((long)p.n_kv * y / ys);
  const int nk = (int)((long)p.n_kv * (y + 1) / ys) - kh0;
  pdl_trigger();
  pdl_wait();
  if (tid < nr) s_slot[tid] = slot_of_row(p, r0 + tid);
  if (__syncthreads_or(list_descends(p))) return;
  if (tid < nr) report_slot(p, s_slot[tid]);
  constexpr int W = DT == DT_MXFP4 ? 16 : 8;
  const int pieces = p.d / W;
  const int L = lanes_for(pieces);
  const int step = kThreads / L;
  const int tensors = p.k_out && p.v_out ? 2 : 1;
  const int nt = tensors * nk;
  // heads outer, rows inner: neighbouring lanes read neighbouring rows
  int h = 0, r = tid / L;
  while (true) {
    while (r >= nr) r -= nr, ++h;
    if (h >= nt) break;
    const long slot = s_slot[r];
    if (slot >= 0) {
      const bool is_v = p.k_out ? h >= nk : true;
      const int hh = kh0 + (h >= nk ? h - nk : h);
      const long row = r0 + r;
      const uint8_t *src = (is_v ? p.v_cache : p.k_cache) +
                           (slot + (long)hh * p.block_size) *
                               row_bytes(p.d, DT);
      uint16_t *dst = is_v ? p.v_out + row * p.vo_rs + hh * p.vo_hs
                           : p.k_out + row * p.ko_rs + hh * p.ko_hs;
      float sc = 1.f;
      if (DT == DT_FP8) sc = (is_v ? p.v_scale : p.k_scale)[hh];
      for (int c = tid & (L - 1); c < pieces; c += L) {
        if constexpr (DT == DT_BF16) {
          *reinterpret_cast<uint4 *>(dst + c * 8) =
              *reinterpret_cast<const uint4 *>(src + c * 16);
        } else if constexpr (DT == DT_FP8) {
          const uint2 u = *reinterpret_cast<const uint2 *>(src + c * 8);
          const uint32_t w[2] = {u.x, u.y};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v =
                e4m3x2_to_f16x2((uint16_t)(w[j >> 1] >> (16 * (j & 1))));
            o[j] = pack_bf16x2(__fmul_rn(f16lo(v), sc),
                               __fmul_rn(f16hi(v), sc));
          }
          *reinterpret_cast<uint4 *>(dst + c * 8) =
              make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          // Words c and c + 8 of the row's 16, so that each store of the lanes
          // fills whole sectors. (Words 2 c and 2 c + 1: 16-byte stores 32
          // bytes apart, of which L2 merges what the compiler happens to put
          // side by side: 24 to 40 million sectors written, 97 to 112 us.)
          uint32_t u[2], g[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            u[j] = *reinterpret_cast<const uint32_t *>(src + 4 * c + 32 * j);
            g[j] = src[64 + (c >> 1) + 4 * j];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t o[4];
            mxfp4_to_bf16(u[j], f16lo(e4m3x2_to_f16x2((uint16_t)g[j])), o);
            reinterpret_cast<uint4 *>(dst)[c + 8 * j] =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
    }
    r += step;
  }
}

// Rows per CTA and head shares: as many rows as keep at least four CTAs per
// SM in the grid (neighbouring rows share cache lines of the cached rows and
// the cost of a CTA's setup); when even single rows leave SMs idle (a decode
// step) each row's heads are shared out as well.
void plan_rows(RowsParams &p, int sms, int max_tile, int max_shares,
               int *shares) {
  p.tile = max_tile;
  while (p.tile > 1 && (p.rows + p.tile - 1) / p.tile < 4 * sms) p.tile /= 2;
  *shares = 1;
  while (*shares * 2 <= max_shares && (long)p.rows * *shares < 2 * sms &&
         p.tile == 1)
    *shares *= 2;
}

template <bool VEC, bool WRITE, int DT>
cudaError_t launch_rows_t(const RowsParams &p, int shares, size_t smem,
                          cudaStream_t s) {
  auto kern = rows_kernel<VEC, WRITE, DT>;
  if (smem > 48 * 1024) {
    static bool done[64] = {};
    const cudaError_t e = set_smem_once(kern, kRowsMaxSmem, done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3((p.rows + p.tile - 1) / p.tile, shares),
                    dim3(kThreads), smem, s, 1, p);
}

template <bool WRITE, int DT>
cudaError_t launch_rows_v(const RowsParams &p, bool vec, int shares,
                          size_t smem, cudaStream_t s) {
  return vec ? launch_rows_t<true, WRITE, DT>(p, shares, smem, s)
             : launch_rows_t<false, WRITE, DT>(p, shares, smem, s);
}

bool vec_ok(const void *ptr, long rs, long hs) {
  return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && rs % 8 == 0 &&
         hs % 8 == 0;
}

// Shared memory of a rows_kernel launch.
size_t rows_smem(const RowsParams &p, bool write, int shares) {
  if (!p.rope.on) return 0;
  size_t b = ((size_t)p.tile * p.rope.half * 8 + 15) / 16 * 16;
  if (write)
    b += (size_t)p.tile * ((p.n_kv + shares - 1) / shares) * p.d * 2;
  return b;
}

}  // namespace

bool rows_fit(int d, int half) {
  return (size_t)half * 8 + 16 + (size_t)d * 2 <= (size_t)kRowsMaxSmem;
}

cudaError_t launch_rows(const RowsParams &in, bool write, int sms,
                        cudaStream_t s) {
  RowsParams p = in;
  if (p.rows == 0) return cudaSuccess;
  int shares = 1;
  const int most = std::max(std::max(p.n_h, p.n_kv), 1);
  plan_rows(p, sms, p.rope.on ? 8 : 16, most, &shares);
  // the turned keys of a CTA in 40 KB, so that five share an SM
  while (p.tile > 1 && rows_smem(p, write, shares) > 40 * 1024) p.tile /= 2;
  while (shares < most && rows_smem(p, write, shares) > 40 * 1024)
    shares = std::min(most, shares * 2);
  const size_t smem = rows_smem(p, write, shares);
  if (smem > (size_t)kRowsMaxSmem || shares > 65535)
    return cudaErrorNotSupported;
  bool vec = true;
  if (p.rope.on) {
    vec = p.d % 8 == 0 && p.d <= 2048 &&
          (p.rope.adjacent ? p.rope.half % 4 == 0 : p.rope.half % 8 == 0);
    if (p.n_h)
      vec = vec && vec_ok(p.q, p.q_rs, p.q_hs) &&
            vec_ok(p.q_out, p.qo_rs, p.qo_hs);
    if (p.n_kv && p.k) vec = vec && vec_ok(p.k, p.k_rs, p.k_hs);
    if (!write && p.n_kv) vec = vec && vec_ok(p.k_out, p.ko_rs, p.ko_hs);
  }
  if (!write) return launch_rows_v<false, DT_BF16>(p, vec, shares, smem, s);
  switch (p.dtype) {
    case DT_BF16: return launch_rows_v<true, DT_BF16>(p, vec, shares, smem, s);
    case DT_FP8: return launch_rows_v<true, DT_FP8>(p, vec, shares, smem, s);
    default: return launch_rows_v<true, DT_MXFP4>(p, vec, shares, smem, s);
  }
}

cudaError_t launch_read(const RowsParams &in, int sms, cudaStream_t s) {
  RowsParams p = in;
  if (p.rows == 0) return cudaSuccess;
  int shares = 1;
  plan_rows(p, sms, kMaxRowTile, p.n_kv, &shares);
  const dim3 grid((p.rows + p.tile - 1) / p.tile, shares);
  switch (p.dtype) {
    case DT_BF16:
      return launch_pdl(read_kernel<DT_BF16>, grid, dim3(kThreads), 0, s, 1,
                        p);
    case DT_FP8:
      return launch_pdl(read_kernel<DT_FP8>, grid, dim3(kThreads), 0, s, 1, p);
    default:
      return launch_pdl(read_kernel<DT_MXFP4>, grid, dim3(kThreads), 0, s, 1,
                        p);
  }
}

}  // namespace kvd
