// The C ABI of libkvd.so (declared in include/kvd.h): host-side argument
// validation, split planning and kernel dispatch. Nothing here allocates
// device memory or synchronises, except kvd_device_error().
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <atomic>
#include <mutex>

#include "kvd.h"
#include "kvd_prompt.h"
#include "kvd_internal.h"
#include "prompt_internal.h"

namespace {

// The library's device error word (one per device that loads the module).
__device__ int g_kvd_device_error;

thread_local char g_msg[512] = "";

kvd_status fail(kvd_status st, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

kvd_status ok() {
  g_msg[0] = 0;
  return KVD_OK;
}

kvd_status cuda_fail(cudaError_t e, const char *what) {
  return fail(KVD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

struct DeviceInfo {
  bool ready = false;
  int sms = 0;
  int *err = nullptr;
};

constexpr int kMaxDevices = 64;
DeviceInfo g_devices[kMaxDevices];
std::mutex g_devices_mu;

// Per-device facts, looked up once per device with that device current.
kvd_status device_info(const DeviceInfo **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices)
    return fail(KVD_ERR_CUDA, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_devices_mu);
  DeviceInfo &d = g_devices[dev];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
    e = cudaGetSymbolAddress(reinterpret_cast<void **>(&d.err),
                             g_kvd_device_error);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress");
    d.ready = true;
  }
  *out = &d;
  return KVD_OK;
}

bool aligned(const void *p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

int env_int(const char *name, int dflt) {
  const char *s = std::getenv(name);
  if (!s || !*s) return dflt;
  return std::atoi(s);
}

// Tuning overrides (kvd_set_tuning): read from the environment once, when
// the library is loaded, and changed only by kvd_set_tuning.
std::atomic<int> g_decode_ctas{env_int("KVD_DECODE_CTAS", 0)};
std::atomic<int> g_mla_cuda_cores{env_int("KVD_MLA_CUDA_CORES", 0)};

// ---------------------------------------------------------------------------
// validation
// ---------------------------------------------------------------------------
kvd_status check_cache(const kvd_cache *c, bool need_v, const char *what) {
  if (!c) return fail(KVD_ERR_NULL, "%s: cache is NULL", what);
  if (!c->k) return fail(KVD_ERR_NULL, "%s: cache->k is NULL", what);
  if (need_v && !c->v)
    return fail(KVD_ERR_NULL, "%s: cache->v is NULL (K and V required)", what);
  if (c->num_blocks < 1 || c->block_size < 1 || c->n_kv < 1 ||
      c->head_dim < 1)
    return fail(KVD_ERR_SHAPE,
                "%s: num_blocks, block_size, n_kv and head_dim must be >= 1",
                what);
  if (c->dtype != KVD_BF16 && c->dtype != KVD_FP8_E4M3 &&
      c->dtype != KVD_MXFP4)
    return fail(KVD_ERR_UNSUPPORTED, "%s: unknown dtype %d", what, c->dtype);
  if (!aligned(c->k, 16) || (c->v && !aligned(c->v, 16)))
    return fail(KVD_ERR_SHAPE, "%s: cache base pointers must be 16-byte aligned",
                what);
  if (c->dtype == KVD_MXFP4) {
    // 72-byte rows, copied two at a time: whole (block, head) runs stay
    // 16-byte multiples when the block size is even
    if (c->head_dim != 128)
      return fail(KVD_ERR_UNSUPPORTED, "%s: mxfp4 caches need head_dim 128",
                  what);
    if (c->block_size % 2 != 0)
      return fail(KVD_ERR_SHAPE, "%s: mxfp4 caches need an even block_size",
                  what);
    return KVD_OK;
  }
  const long row_bytes =
      (long)c->head_dim * (c->dtype == KVD_BF16 ? 2 : 1);
  if (row_bytes % 16 != 0)
    return fail(KVD_ERR_SHAPE, "%s: a cache row (%ld bytes) must be a multiple "
                "of 16 bytes", what, row_bytes);
  return KVD_OK;
}

// Calls other than the dense GQA decode attend to every position they are
// given: a sliding window there is refused.
kvd_status no_window(const kvd_seqs *s, const char *what) {
  if (s && (s->window != 0 || s->window_start))
    return fail(KVD_ERR_UNSUPPORTED, "%s: no sliding window (window and "
                "window_start are for the GQA decode calls)", what);
  return KVD_OK;
}

kvd_status check_seqs(const kvd_seqs *s, const kvd_cache *c, const char *what) {
  if (!s) return fail(KVD_ERR_NULL, "%s: seqs is NULL", what);
  if (s->batch < 0 || s->max_blocks_per_seq < 1 || s->max_seq_len < 0)
    return fail(KVD_ERR_SHAPE,
                "%s: batch >= 0, max_blocks_per_seq >= 1, max_seq_len >= 0 "
                "required", what);
  if (s->batch > 65535)
    return fail(KVD_ERR_SHAPE, "%s: batch %d above 65535", what, s->batch);
  if (s->flags & ~(KVD_SEQS_STABLE | KVD_SEQS_PREFIX_READY))
    return fail(KVD_ERR_SHAPE, "%s: unknown seqs flags 0x%x", what,
                (unsigned)s->flags);
  if ((s->flags & KVD_SEQS_PREFIX_READY) && !(s->flags & KVD_SEQS_STABLE))
    return fail(KVD_ERR_SHAPE, "%s: KVD_SEQS_PREFIX_READY needs "
                "KVD_SEQS_STABLE", what);
  if (s->batch > 0 && (!s->block_table || !s->seq_lens))
    return fail(KVD_ERR_NULL, "%s: block_table and seq_lens are required", what);
  if (s->window < 0)
    return fail(KVD_ERR_SHAPE, "%s: window must be >= 0", what);
  if ((long)s->max_seq_len > (long)s->max_blocks_per_seq * c->block_size)
    return fail(KVD_ERR_CAPACITY,
                "%s: max_seq_len %d exceeds the block table's capacity %ld",
                what, s->max_seq_len,
                (long)s->max_blocks_per_seq * c->block_size);
  return KVD_OK;
}

// ---------------------------------------------------------------------------
// split plans
// ---------------------------------------------------------------------------
struct Plan {
  int split_len = kvd::kStageRows;
  int n_splits = 1;
  int n_groups = 1;        // head groups (tiles) per sequence
  size_t ws_o_bytes = 0;   // partial outputs
  size_t ws_lse_bytes = 0; // partial log-sum-exps
  size_t ws_bytes = 0;     // total
  int hp = 1;              // kv heads per work unit (CUDA-core GQA kernel)
  int whole_units = 0;     // dense GQA: one CTA per unit, no merge
  int cluster = 0;         // dense GQA: CTAs per unit of a cluster merge
};

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

enum class DenseKernel { Simt, Mma };

kvd_status gqa_shape(const kvd_cache *c, int n_h, DenseKernel *kind) {
  if (n_h < 1 || n_h % c->n_kv != 0)
    return fail(KVD_ERR_SHAPE, "gqa_decode: n_h (%d) must be a positive "
                "multiple of n_kv (%d)", n_h, c->n_kv);
  const int g = n_h / c->n_kv;
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(KVD_ERR_UNSUPPORTED, "gqa_decode: head_dim %d (64 or 128)",
                c->head_dim);
  if (c->dtype == KVD_MXFP4 && g != 1 && g != 2 && g != 4)
    return fail(KVD_ERR_UNSUPPORTED, "gqa_decode: mxfp4 caches are decoded "
                "on the CUDA-core kernel: group size 1, 2 or 4 (got %d)", g);
  if (g == 1 || g == 2 || g == 4) {
    *kind = DenseKernel::Simt;
  } else if ((g == 8 || g == 16) && c->head_dim == 128) {
    *kind = DenseKernel::Mma;
  } else {
    return fail(KVD_ERR_UNSUPPORTED,
                "gqa_decode: group size %d with head_dim %d", g, c->head_dim);
  }
  return KVD_OK;
}

// Units (sequence, head group) of at most this many 64-token chunks run one
// per CTA when they fit in one wave: the merge launch and its two grid
// dependencies (about 3 us) then cost more than the imbalance of whole
// units (at most this many chunks against the average share).
constexpr int kWholeUnitChunks = 4;

// Persistent stream-K plan of the dense GQA kernels: `ctas_per_sm` CTAs per
// SM (never more CTAs than 64-token chunks), each leaving at most two
// partials of G heads x head_dim, which the merge launch combines. Short
// units instead run whole, one CTA each (no partials, no merge): every unit
// holds at most kWholeUnitChunks chunks (the window bounds it, or the
// longest visible length does) and there are no more units than CTAs.
Plan plan_stream_k(int sms, int ctas_per_sm, int batch, int n_kv, int g,
                   int d, int max_seq_len, int window = 0) {
  Plan pl;
  const int R = kvd::kStageRows;
  const long unit_chunks =
      window > 0 ? std::min<long>((window + R - 1) / R + 1,
                                  (max_seq_len + R - 1) / R)
                 : (max_seq_len + R - 1) / R;
  const long chunks = (long)batch * n_kv * ((max_seq_len + R - 1) / R);
  long ctas = (long)sms * ctas_per_sm;
  const int forced = g_decode_ctas.load(std::memory_order_relaxed);
  const long units = (long)batch * n_kv;
  if (forced <= 0 && units >= 1 && units <= ctas &&
      unit_chunks <= kWholeUnitChunks) {
    pl.whole_units = 1;
    pl.n_splits = (int)units;
    pl.n_groups = n_kv;
    return pl;  // no workspace
  }
  if (forced > 0) ctas = forced;
  ctas = std::max(1L, std::min(ctas, std::max(chunks, 1L)));
  pl.n_splits = (int)ctas;
  pl.n_groups = n_kv;
  pl.ws_o_bytes = round_up((size_t)ctas * 2 * g * d * 4, 256);
  pl.ws_lse_bytes = round_up((size_t)ctas * 2 * g * 4, 256);
  pl.ws_bytes = pl.ws_o_bytes + pl.ws_lse_bytes;
  return pl;
}

Plan gqa_plan(const kvd_cache *c, const kvd_seqs *s, int n_h, int sms,
              DenseKernel kind) {
  const int g = n_h / c->n_kv;
  const int hp = kind == DenseKernel::Simt
                     ? kvd::simt_heads_per_stage(c->n_kv, g, c->head_dim,
                                                 c->dtype, c->block_size)
                     : kvd::mma_heads_per_unit(c->n_kv, c->block_size,
                                               c->dtype);
  Plan pl = plan_stream_k(sms, 1, s->batch, c->n_kv / hp, g * hp,
                          c->head_dim, s->max_seq_len, s->window);
  pl.hp = hp;
  // One sequence (every unit as long as the others) on the CUDA-core
  // kernel with query groups of 1: its units run as clusters of CTAs that
  // merge their parts in distributed shared memory, when all the clusters
  // fit at once -- no workspace and no merge launch.
  if (kind == DenseKernel::Simt && !pl.whole_units && s->batch == 1 &&
      g == 1 && g_decode_ctas.load(std::memory_order_relaxed) <= 0) {
    const int units = c->n_kv / hp;
    const int cs =
        kvd::simt_cluster_size(c->head_dim, c->dtype, hp, units, sms);
    if (cs >= 2) {
      Plan cl;
      cl.cluster = cs;
      cl.n_splits = units * cs;
      cl.n_groups = units;
      cl.hp = hp;
      return cl;
    }
  }
  return pl;
}

// Persistent stream-K plan of the latent decode kernels: 32-position (or
// 64-position) chunks of `rows` positions per sequence and head tile;
// partials of 64 heads x dv per CTA side, merged by a second launch.
// `per_lane` CTAs of the launch share a lane's chunk range (one per head
// tile, or per head tile and value part for the tensor-core latent
// kernel); n_splits counts 64-head tiles per lane whatever the kernel.
Plan plan_wide(int sms, int batch, int n_h, int rows, int dv,
               int per_lane = 0, int chunk_rows = 32) {
  Plan pl;
  const int tiles = n_h / 64;
  if (per_lane <= 0) per_lane = tiles;
  const long chunks = (long)batch * ((rows + chunk_rows - 1) / chunk_rows);
  long ctas = sms;
  const int forced = g_decode_ctas.load(std::memory_order_relaxed);
  if (forced > 0) ctas = forced;
  const long lanes =
      std::max(1L, std::min(ctas / per_lane, std::max(chunks, 1L)));
  ctas = lanes * tiles;
  pl.n_splits = (int)ctas;
  pl.n_groups = tiles;
  pl.ws_o_bytes = round_up((size_t)ctas * 2 * 64 * dv * 4, 256);
  pl.ws_lse_bytes = round_up((size_t)ctas * 2 * 64 * 4, 256);
  pl.ws_bytes = pl.ws_o_bytes + pl.ws_lse_bytes;
  return pl;
}

// The latent decode runs on the tcgen05 kernel where its shape allows
// (kvd_set_tuning can select the CUDA-core kernel everywhere).
bool mla_on_tensor_memory(const kvd_cache *c, int n_h) {
  return g_mla_cuda_cores.load(std::memory_order_relaxed) == 0 &&
         kvd::latent_tc_supported(n_h, c->block_size, c->num_blocks);
}

Plan mla_plan(const kvd_seqs *s, int n_h, int dv, int sms, bool tc) {
  return tc ? plan_wide(sms, s->batch, n_h, s->max_seq_len, dv,
                       n_h / 128 * kvd::kLatentTcParts,
                       kvd::kLatentTcRows)
            : plan_wide(sms, s->batch, n_h, s->max_seq_len, dv);
}

// The tcgen05 gather kernel: S CTAs per (sequence, 64-head tile), one
// wave. With S > 1 each CTA leaves its part (64 heads x 512 values fp32 +
// 64 lse) for the merge launch.
Plan sparse_plan(const kvd_seqs *s, int n_h, int k, int dv, int sms) {
  Plan pl;
  const int units = std::max(s->batch * (n_h / 64), 1);
  const int S = kvd::gather_tc_splits(
      units, std::max(k, 1), sms, g_decode_ctas.load(std::memory_order_relaxed));
  pl.n_splits = S;
  pl.n_groups = 1;
  const size_t slots = (size_t)units * S;
  pl.ws_o_bytes = S > 1 ? round_up(slots * 64 * dv * 4, 256) : 0;
  pl.ws_lse_bytes = S > 1 ? round_up(slots * 64 * 4, 256) : 0;
  pl.ws_bytes = pl.ws_o_bytes + pl.ws_lse_bytes;
  return pl;
}

size_t topk_ws_bytes(const kvd_seqs *s) {
  return round_up((size_t)s->batch * std::max(s->max_seq_len, 1) * 4, 256);
}

kvd_status check_ws(const Plan &pl, void *ws, size_t bytes, const char *what) {
  if (pl.ws_bytes == 0) return KVD_OK;
  if (!ws)
    return fail(KVD_ERR_WORKSPACE, "%s: workspace of %zu bytes required", what,
                pl.ws_bytes);
  if (!aligned(ws, 256))
    return fail(KVD_ERR_WORKSPACE, "%s: workspace must be 256-byte aligned",
                what);
  if (bytes < pl.ws_bytes)
    return fail(KVD_ERR_WORKSPACE, "%s: workspace %zu < required %zu bytes",
                what, bytes, pl.ws_bytes);
  return KVD_OK;
}

float log2_scale(float scale, int dk) {
  const float s = scale > 0.f ? scale : 1.0f / std::sqrt((float)dk);
  return s * 1.4426950408889634f;
}

kvd_status launched(cudaError_t e, const char *what) {
  if (e == cudaErrorNotSupported)
    return fail(KVD_ERR_UNSUPPORTED, "%s: kernel not available", what);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return ok();
}

}  // namespace

namespace kvd {
namespace {
std::atomic<unsigned long long> g_launches{0};
}  // namespace

void note_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }

// Workspace bytes of a gqa_decode call with these arguments on the current
// device (validating them as the call does). Used by the no-allocation entry
// point.
kvd_status gqa_workspace_bytes(const kvd_cache *cache, const kvd_seqs *seqs,
                               int32_t n_h, size_t *total) {
  kvd_status st = check_cache(cache, true, "gqa_decode");
  if (st != KVD_OK) return st;
  st = check_seqs(seqs, cache, "gqa_decode");
  if (st != KVD_OK) return st;
  DenseKernel kind;
  st = gqa_shape(cache, n_h, &kind);
  if (st != KVD_OK) return st;
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  *total = gqa_plan(cache, seqs, n_h, d->sms, kind).ws_bytes;
  return KVD_OK;
}

kvd_status device_error_word(int **err) {
  const DeviceInfo *d = nullptr;
  const kvd_status st = device_info(&d);
  if (st != KVD_OK) return st;
  *err = d->err;
  return KVD_OK;
}

kvd_status set_error(kvd_status st, const char *msg) {
  return fail(st, "%s", msg);
}
}  // namespace kvd

// ===========================================================================
// C ABI
// ===========================================================================
extern "C" {

int32_t kvd_version(void) { return KVD_VERSION; }

kvd_status kvd_set_tuning(int32_t decode_ctas, int32_t mla_cuda_cores) {
  if (decode_ctas < 0)
    return fail(KVD_ERR_SHAPE, "set_tuning: decode_ctas must be >= 0");
  g_decode_ctas.store(decode_ctas, std::memory_order_relaxed);
  g_mla_cuda_cores.store(mla_cuda_cores != 0, std::memory_order_relaxed);
  return ok();
}

uint64_t kvd_launch_count(void) {
  return kvd::g_launches.load(std::memory_order_relaxed);
}

const char *kvd_last_error(void) { return g_msg; }

const char *kvd_status_string(kvd_status st) {
  switch (st) {
    case KVD_OK: return "KVD_OK";
    case KVD_ERR_NULL: return "KVD_ERR_NULL";
    case KVD_ERR_SHAPE: return "KVD_ERR_SHAPE";
    case KVD_ERR_UNSUPPORTED: return "KVD_ERR_UNSUPPORTED";
    case KVD_ERR_CAPACITY: return "KVD_ERR_CAPACITY";
    case KVD_ERR_WORKSPACE: return "KVD_ERR_WORKSPACE";
    case KVD_ERR_CUDA: return "KVD_ERR_CUDA";
  }
  return "KVD_ERR_UNKNOWN";
}

uint64_t kvd_bytes_per_token(int32_t n_l, int32_t n_kv, int32_t d_h,
                             int32_t elem_bytes) {
  if (n_l < 0 || n_kv < 0 || d_h < 0 || elem_bytes < 0) return 0;
  return 2ull * (uint64_t)n_l * (uint64_t)n_kv * (uint64_t)d_h *
         (uint64_t)elem_bytes;
}

kvd_status kvd_device_error(int32_t *code) {
  if (!code) return fail(KVD_ERR_NULL, "device_error: code is NULL");
  const DeviceInfo *d = nullptr;
  kvd_status st = device_info(&d);
  if (st != KVD_OK) return st;
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
  int v = 0;
  e = cudaMemcpy(&v, d->err, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return cuda_fail(e, "read device error word");
  const int zero = 0;
  e = cudaMemcpy(d->err, &zero, sizeof(int), cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return cuda_fail(e, "clear device error word");
  *code = v;
  return ok();
}

kvd_status kvd_kv_append(const kvd_cache *cache, const int32_t *block_table,
                         int32_t max_blocks_per_seq, const int32_t *pos,
                         int32_t batch, const void *k_new, const void *v_new,
                         kvd_stream stream) {
  kvd_status st = check_cache(cache, false, "kv_append");
  if (st != KVD_OK) return st;
  if (batch < 0 || batch > 65535 || max_blocks_per_seq < 1)
    return fail(KVD_ERR_SHAPE, "kv_append: 0 <= batch <= 65535 and "
                "max_blocks_per_seq >= 1 required");
  if (cache->head_dim % 8 != 0)
    return fail(KVD_ERR_SHAPE, "kv_append: head_dim must be a multiple of 8");
  if (batch == 0) return ok();
  if (!block_table || !pos || !k_new)
    return fail(KVD_ERR_NULL, "kv_append: block_table, pos and k_new required");
  if (cache->v && !v_new)
    return fail(KVD_ERR_NULL, "kv_append: v_new required for a K/V cache");
  if (!aligned(k_new, 16) || (cache->v && !aligned(v_new, 16)))
    return fail(KVD_ERR_SHAPE, "kv_append: k_new / v_new must be 16-byte "
                "aligned");
  if (cache->dtype == KVD_FP8_E4M3 &&
      (!cache->k_inv_scale || (cache->v && !cache->v_inv_scale)))
    return fail(KVD_ERR_NULL, "kv_append: fp8 cache needs inverse scales");
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  kvd::AppendParams p{};
  p.k_cache = static_cast<uint8_t *>(cache->k);
  p.v_cache = static_cast<uint8_t *>(cache->v);
  p.k_inv_scale = cache->k_inv_scale;
  p.v_inv_scale = cache->v_inv_scale;
  p.block_table = block_table;
  p.pos = pos;
  p.k_new = static_cast<const uint16_t *>(k_new);
  p.v_new = static_cast<const uint16_t *>(v_new);
  p.num_blocks = cache->num_blocks;
  p.block_size = cache->block_size;
  p.n_kv = cache->n_kv;
  p.head_dim = cache->head_dim;
  p.dtype = cache->dtype;
  p.max_blocks = max_blocks_per_seq;
  p.batch = batch;
  p.err = d->err;
  return launched(kvd::launch_append(p, reinterpret_cast<cudaStream_t>(stream)),
                  "kv_append");
}

kvd_status kvd_workspace_size(kvd_op op, const kvd_cache *cache,
                              const kvd_seqs *seqs, int32_t n_h, int32_t k,
                              size_t *bytes) {
  if (!bytes) return fail(KVD_ERR_NULL, "workspace_size: bytes is NULL");
  kvd_status st = check_cache(cache, false, "workspace_size");
  if (st != KVD_OK) return st;
  st = check_seqs(seqs, cache, "workspace_size");
  if (st != KVD_OK) return st;
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  switch (op) {
    case KVD_OP_GQA_DECODE: {
      DenseKernel kind;
      st = gqa_shape(cache, n_h, &kind);
      if (st != KVD_OK) return st;
      *bytes = gqa_plan(cache, seqs, n_h, d->sms, kind).ws_bytes;
      return ok();
    }
    case KVD_OP_MLA_DECODE:
      if (n_h < 64 || n_h % 64 != 0)
        return fail(KVD_ERR_UNSUPPORTED, "mla: n_h must be a multiple of 64");
      *bytes = mla_plan(seqs, n_h, 512, d->sms,
                        mla_on_tensor_memory(cache, n_h)).ws_bytes;
      return ok();
    case KVD_OP_SPARSE_DECODE:
      if (n_h < 64 || n_h % 64 != 0 || k < 1)
        return fail(KVD_ERR_UNSUPPORTED,
                    "sparse: n_h must be a multiple of 64 and k >= 1");
      *bytes = sparse_plan(seqs, n_h, k, cache->head_dim, d->sms).ws_bytes;
      return ok();
    case KVD_OP_INDEXER_TOPK:
      *bytes = topk_ws_bytes(seqs);
      return ok();
    case KVD_OP_INDEXER_TOPK_POOL:
      *bytes = round_up((size_t)seqs->batch * kvd::kPoolBlocks *
                            kvd::kPoolBlock * 4, 256);
      return ok();
  }
  return fail(KVD_ERR_UNSUPPORTED, "workspace_size: unknown op %d", (int)op);
}

}  // extern "C"

namespace {
// kvd_gqa_decode, and kvd_gqa_append_decode when pos != nullptr.
kvd_status gqa_decode_impl(const kvd_cache *cache, const kvd_seqs *seqs,
                           const int32_t *pos, const void *k_new,
                           const void *v_new, const void *q, int32_t n_h,
                           float scale, void *out, float *lse,
                           void *workspace, size_t workspace_bytes,
                           kvd_stream stream) {
  kvd_status st = check_cache(cache, true, "gqa_decode");
  if (st != KVD_OK) return st;
  st = check_seqs(seqs, cache, "gqa_decode");
  if (st != KVD_OK) return st;
  DenseKernel kind;
  st = gqa_shape(cache, n_h, &kind);
  if (st != KVD_OK) return st;
  if (seqs->batch > 1024)
    return fail(KVD_ERR_UNSUPPORTED, "gqa_decode: at most 1024 sequences "
                "per call (got %d)", seqs->batch);
  if (cache->dtype == KVD_FP8_E4M3 && (!cache->k_scale || !cache->v_scale))
    return fail(KVD_ERR_NULL, "gqa_decode: fp8 cache needs k_scale, v_scale");
  if (seqs->batch == 0) return ok();
  if (!q || !out) return fail(KVD_ERR_NULL, "gqa_decode: q and out required");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(KVD_ERR_SHAPE, "gqa_decode: q and out must be 16-byte aligned");
  if (pos) {
    if (!k_new || !v_new)
      return fail(KVD_ERR_NULL, "gqa_append_decode: k_new and v_new required");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
      return fail(KVD_ERR_SHAPE, "gqa_append_decode: k_new / v_new must be "
                  "16-byte aligned");
    if (cache->dtype == KVD_FP8_E4M3 &&
        (!cache->k_inv_scale || !cache->v_inv_scale))
      return fail(KVD_ERR_NULL,
                  "gqa_append_decode: fp8 cache needs inverse scales");
  }
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  const Plan pl = gqa_plan(cache, seqs, n_h, d->sms, kind);
  st = check_ws(pl, workspace, workspace_bytes, "gqa_decode");
  if (st != KVD_OK) return st;

  kvd::DecodeParams p{};
  p.k = static_cast<const uint8_t *>(cache->k);
  p.v = static_cast<const uint8_t *>(cache->v);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.block_table = seqs->block_table;
  p.seq_lens = seqs->seq_lens;
  p.q = static_cast<const uint16_t *>(q);
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                       pl.ws_o_bytes);
  p.n_groups = pl.n_groups;
  p.batch = seqs->batch;
  p.n_h = n_h;
  p.n_kv = cache->n_kv;
  p.dk = p.dv = cache->head_dim;
  p.dtype = cache->dtype;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.max_blocks = seqs->max_blocks_per_seq;
  p.max_seq_len = seqs->max_seq_len;
  p.split_len = pl.split_len;
  p.n_splits = pl.n_splits;
  p.whole_units = pl.whole_units;
  p.cluster = pl.cluster;
  p.hp = pl.hp;
  p.flags = seqs->flags;
  p.window = seqs->window;
  p.win_start = seqs->window_start;
  p.pos = pos;
  p.k_new = static_cast<const uint16_t *>(k_new);
  p.v_new = static_cast<const uint16_t *>(v_new);
  p.k_inv_scale = cache->k_inv_scale;
  p.v_inv_scale = cache->v_inv_scale;
  p.scale_log2 = log2_scale(scale, cache->head_dim);
  p.err = d->err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = kind == DenseKernel::Simt
                      ? kvd::launch_decode_simt(p, s)
                      : kvd::launch_decode_mma(p, cache->dtype, s);
  return launched(e, "gqa_decode");
}
}  // namespace


extern "C" {

kvd_status kvd_gqa_decode(const kvd_cache *cache, const kvd_seqs *seqs,
                          const void *q, int32_t n_h, float scale, void *out,
                          float *lse, void *workspace, size_t workspace_bytes,
                          kvd_stream stream) {
  return gqa_decode_impl(cache, seqs, nullptr, nullptr, nullptr, q, n_h, scale,
                         out, lse, workspace, workspace_bytes, stream);
}

kvd_status kvd_gqa_append_decode(const kvd_cache *cache, const kvd_seqs *seqs,
                                 const int32_t *pos, const void *k_new,
                                 const void *v_new, const void *q, int32_t n_h,
                                 float scale, void *out, float *lse,
                                 void *workspace, size_t workspace_bytes,
                                 kvd_stream stream) {
  if (!pos && seqs && seqs->batch > 0)
    return fail(KVD_ERR_NULL, "gqa_append_decode: pos required");
  return gqa_decode_impl(cache, seqs, pos, k_new, v_new, q, n_h, scale, out,
                         lse, workspace, workspace_bytes, stream);
}

kvd_status kvd_mla_decode(const kvd_cache *latent, int32_t d_c,
                          const kvd_seqs *seqs, const void *q, int32_t n_h,
                          float scale, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, kvd_stream stream) {
  kvd_status st = check_cache(latent, false, "mla_decode");
  if (st != KVD_OK) return st;
  st = check_seqs(seqs, latent, "mla_decode");
  if (st != KVD_OK) return st;
  st = no_window(seqs, "mla_decode");
  if (st != KVD_OK) return st;
  if (latent->dtype != KVD_BF16 || latent->n_kv != 1 || d_c != 512 ||
      latent->head_dim != 576)
    return fail(KVD_ERR_UNSUPPORTED, "mla_decode: bf16 latent cache with "
                "n_kv = 1, d_c = 512, head_dim = 576 required");
  if (n_h < 64 || n_h % 64 != 0)
    return fail(KVD_ERR_UNSUPPORTED, "mla_decode: n_h must be a multiple of 64");
  if (seqs->batch > 256)
    return fail(KVD_ERR_UNSUPPORTED, "mla_decode: at most 256 sequences");
  if (seqs->batch == 0) return ok();
  if (!q || !out) return fail(KVD_ERR_NULL, "mla_decode: q and out required");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(KVD_ERR_SHAPE, "mla_decode: q and out must be 16-byte aligned");
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  const bool tc = mla_on_tensor_memory(latent, n_h);
  const Plan pl = mla_plan(seqs, n_h, d_c, d->sms, tc);
  st = check_ws(pl, workspace, workspace_bytes, "mla_decode");
  if (st != KVD_OK) return st;
  kvd::DecodeParams p{};
  p.k = p.v = static_cast<const uint8_t *>(latent->k);
  p.block_table = seqs->block_table;
  p.seq_lens = seqs->seq_lens;
  p.q = static_cast<const uint16_t *>(q);
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                       pl.ws_o_bytes);
  p.n_groups = pl.n_groups;
  p.batch = seqs->batch;
  p.n_h = n_h;
  p.n_kv = 1;
  p.dk = latent->head_dim;
  p.dv = d_c;
  p.block_size = latent->block_size;
  p.num_blocks = latent->num_blocks;
  p.max_blocks = seqs->max_blocks_per_seq;
  p.max_seq_len = seqs->max_seq_len;
  p.split_len = pl.split_len;
  p.n_splits = pl.n_splits;
  p.scale_log2 = log2_scale(scale, latent->head_dim);
  p.err = d->err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(tc ? kvd::launch_decode_mla_tc(p, s)
                     : kvd::launch_decode_mla(p, s),
                  "mla_decode");
}

kvd_status kvd_sparse_decode(const kvd_cache *cache, const kvd_seqs *seqs,
                             const int32_t *indices, int32_t k, const void *q,
                             int32_t n_h, float scale, void *out, float *lse,
                             void *workspace, size_t workspace_bytes,
                             kvd_stream stream) {
  kvd_status st = check_cache(cache, true, "sparse_decode");
  if (st != KVD_OK) return st;
  st = check_seqs(seqs, cache, "sparse_decode");
  if (st != KVD_OK) return st;
  st = no_window(seqs, "sparse_decode");
  if (st != KVD_OK) return st;
  if (cache->dtype != KVD_BF16 || cache->n_kv != 1 || cache->head_dim != 512)
    return fail(KVD_ERR_UNSUPPORTED, "sparse_decode: bf16 cache with n_kv = 1 "
                "and head_dim = 512 required");
  if (n_h < 64 || n_h % 64 != 0)
    return fail(KVD_ERR_UNSUPPORTED,
                "sparse_decode: n_h must be a multiple of 64");
  if (k < 1) return fail(KVD_ERR_SHAPE, "sparse_decode: k must be >= 1");
  if (seqs->batch > 256)
    return fail(KVD_ERR_UNSUPPORTED, "sparse_decode: at most 256 sequences");
  if (seqs->batch == 0) return ok();
  if (!indices || !q || !out)
    return fail(KVD_ERR_NULL, "sparse_decode: indices, q and out required");
  if (!aligned(q, 16) || !aligned(out, 16))
    return fail(KVD_ERR_SHAPE, "sparse_decode: q and out must be 16-byte "
                "aligned");
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  const Plan pl = sparse_plan(seqs, n_h, k, cache->head_dim, d->sms);
  st = check_ws(pl, workspace, workspace_bytes, "sparse_decode");
  if (st != KVD_OK) return st;
  kvd::DecodeParams p{};
  p.k = static_cast<const uint8_t *>(cache->k);
  p.v = static_cast<const uint8_t *>(cache->v);
  p.block_table = seqs->block_table;
  p.seq_lens = seqs->seq_lens;
  p.indices = indices;
  p.q = static_cast<const uint16_t *>(q);
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                       pl.ws_o_bytes);
  p.n_groups = pl.n_groups;
  p.batch = seqs->batch;
  p.n_h = n_h;
  p.n_kv = 1;
  p.dk = p.dv = cache->head_dim;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.max_blocks = seqs->max_blocks_per_seq;
  p.max_seq_len = seqs->max_seq_len;
  p.n_idx = k;
  p.split_len = pl.split_len;
  p.n_splits = pl.n_splits;
  p.scale_log2 = log2_scale(scale, cache->head_dim);
  p.err = d->err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(kvd::launch_decode_sparse_tc(p, s), "sparse_decode");
}

}  // extern "C"

namespace {

// kvd_indexer_topk and (pool != NULL) kvd_indexer_topk_pool.
kvd_status indexer_topk_impl(const kvd_cache *index_cache,
                             const kvd_seqs *seqs, const void *q_idx,
                             int32_t n_idx_heads, const float *w,
                             const int32_t *pool, const int32_t *pool_n,
                             int32_t k, int32_t *indices, float *scores,
                             void *workspace, size_t workspace_bytes,
                             kvd_stream stream) {
  kvd_status st = check_cache(index_cache, false, "indexer_topk");
  if (st != KVD_OK) return st;
  st = check_seqs(seqs, index_cache, "indexer_topk");
  if (st != KVD_OK) return st;
  st = no_window(seqs, "indexer_topk");
  if (st != KVD_OK) return st;
  if (index_cache->dtype != KVD_BF16 || index_cache->n_kv != 1 ||
      index_cache->head_dim != 64)
    return fail(KVD_ERR_UNSUPPORTED, "indexer_topk: bf16 K-only cache with "
                "n_kv = 1 and head_dim = 64 required");
  if (n_idx_heads < 1 || n_idx_heads > 8)
    return fail(KVD_ERR_UNSUPPORTED, "indexer_topk: 1..8 indexer heads");
  if (k < 1 || k > 16384)
    return fail(KVD_ERR_UNSUPPORTED, "indexer_topk: k must be in [1, 16384]");
  if (pool && index_cache->block_size % kvd::kPoolBlock != 0)
    return fail(KVD_ERR_UNSUPPORTED, "indexer_topk_pool: block_size must be "
                "a multiple of 8");
  if (seqs->batch == 0) return ok();
  if (!q_idx || !w || !indices)
    return fail(KVD_ERR_NULL, "indexer_topk: q_idx, w and indices required");
  if (pool && !pool_n)
    return fail(KVD_ERR_NULL, "indexer_topk_pool: pool and pool_n required");
  if (!aligned(q_idx, 16))
    return fail(KVD_ERR_SHAPE, "indexer_topk: q_idx must be 16-byte aligned");
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  const int entries = pool ? kvd::kPoolBlocks * kvd::kPoolBlock
                           : seqs->max_seq_len;
  float *sc = scores;
  if (!sc) {
    const size_t need =
        pool ? round_up((size_t)seqs->batch * entries * 4, 256)
             : topk_ws_bytes(seqs);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need)
      return fail(KVD_ERR_WORKSPACE, "indexer_topk: workspace of %zu bytes "
                  "(256-byte aligned) required when scores is NULL", need);
    sc = static_cast<float *>(workspace);
  }
  kvd::IndexerParams p{};
  p.cache = static_cast<const uint8_t *>(index_cache->k);
  p.block_table = seqs->block_table;
  p.seq_lens = seqs->seq_lens;
  p.q = static_cast<const uint16_t *>(q_idx);
  p.w = w;
  p.scores = sc;
  p.indices = indices;
  p.batch = seqs->batch;
  p.n_heads = n_idx_heads;
  p.block_size = index_cache->block_size;
  p.num_blocks = index_cache->num_blocks;
  p.max_blocks = seqs->max_blocks_per_seq;
  p.max_seq_len = seqs->max_seq_len;
  p.score_stride = std::max(entries, 1);
  p.topk = k;
  p.pool = pool;
  p.pool_n = pool_n;
  p.max_entries = entries;
  p.flags = seqs->flags;
  p.err = d->err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = launched(kvd::launch_indexer_scores(p, s), "indexer_topk (scores)");
  if (st != KVD_OK) return st;
  return launched(kvd::launch_topk(p, s), "indexer_topk (select)");
}

}  // namespace

extern "C" {

kvd_status kvd_indexer_topk(const kvd_cache *index_cache, const kvd_seqs *seqs,
                            const void *q_idx, int32_t n_idx_heads,
                            const float *w, int32_t k, int32_t *indices,
                            float *scores, void *workspace,
                            size_t workspace_bytes, kvd_stream stream) {
  return indexer_topk_impl(index_cache, seqs, q_idx, n_idx_heads, w, nullptr,
                           nullptr, k, indices, scores, workspace,
                           workspace_bytes, stream);
}

kvd_status kvd_indexer_topk_pool(const kvd_cache *index_cache,
                                 const kvd_seqs *seqs, const void *q_idx,
                                 int32_t n_idx_heads, const float *w,
                                 const int32_t *pool, const int32_t *pool_n,
                                 int32_t k, int32_t *indices, float *scores,
                                 void *workspace, size_t workspace_bytes,
                                 kvd_stream stream) {
  if (!pool)
    return fail(KVD_ERR_NULL, "indexer_topk_pool: pool required");
  return indexer_topk_impl(index_cache, seqs, q_idx, n_idx_heads, w, pool,
                           pool_n, k, indices, scores, workspace,
                           workspace_bytes, stream);
}

kvd_status kvd_indexer_pool(const kvd_seqs *seqs, const int32_t *indices,
                            int32_t k, int32_t *pool, int32_t *pool_n,
                            kvd_stream stream) {
  if (!seqs) return fail(KVD_ERR_NULL, "indexer_pool: seqs is NULL");
  if (seqs->batch < 0 || seqs->batch > 65535 || seqs->max_seq_len < 0)
    return fail(KVD_ERR_SHAPE, "indexer_pool: 0 <= batch <= 65535 and "
                "max_seq_len >= 0 required");
  if (k < 1) return fail(KVD_ERR_SHAPE, "indexer_pool: k must be >= 1");
  kvd_status wst = no_window(seqs, "indexer_pool");
  if (wst != KVD_OK) return wst;
  if ((long)seqs->max_seq_len > 50331648L)
    return fail(KVD_ERR_UNSUPPORTED, "indexer_pool: max_seq_len above "
                "50,331,648");
  if (seqs->batch == 0) return ok();
  if (!seqs->seq_lens || !indices || !pool || !pool_n)
    return fail(KVD_ERR_NULL, "indexer_pool: seq_lens, indices, pool and "
                "pool_n required");
  const DeviceInfo *d = nullptr;
  kvd_status st = device_info(&d);
  if (st != KVD_OK) return st;
  kvd::PoolParams p{};
  p.indices = indices;
  p.seq_lens = seqs->seq_lens;
  p.pool = pool;
  p.pool_n = pool_n;
  p.batch = seqs->batch;
  p.k = k;
  p.max_seq_len = seqs->max_seq_len;
  p.err = d->err;
  return launched(kvd::launch_indexer_pool(
                      p, reinterpret_cast<cudaStream_t>(stream)),
                  "indexer_pool");
}

}  // extern "C"

// ===========================================================================
// the prompt path (kvd_prompt.h)
// ===========================================================================
namespace {

// Rows of a ragged tensor: `out` ones may not overlap one another.
kvd_status check_rows(const kvd_rows *r, int d, bool out, const char *what,
                      const char *name) {
  if (r->rows < 0 || r->heads < 1)
    return fail(KVD_ERR_SHAPE, "%s: %s needs rows >= 0 and heads >= 1", what,
                name);
  if (r->rows > 0 && !r->data)
    return fail(KVD_ERR_NULL, "%s: %s->data is NULL", what, name);
  if (!aligned(r->data, 2))
    return fail(KVD_ERR_SHAPE, "%s: %s->data is not 2-byte aligned", what,
                name);
  const int64_t lim = int64_t(1) << 40;
  if (r->row_stride < 0 || r->head_stride < 0 || r->row_stride > lim ||
      r->head_stride > lim)
    return fail(KVD_ERR_SHAPE, "%s: %s strides must be in [0, 2^40]", what,
                name);
  if (!out) return KVD_OK;
  const int64_t rs = r->row_stride, hs = r->head_stride;
  const bool heads_fit = r->heads == 1 || hs >= d;
  const bool rows_fit = r->rows <= 1 || rs >= d;
  const bool apart = r->heads == 1 || r->rows <= 1 ||
                     rs >= (int64_t)(r->heads - 1) * hs + d ||
                     hs >= (int64_t)(r->rows - 1) * rs + d;
  if (!heads_fit || !rows_fit || !apart)
    return fail(KVD_ERR_SHAPE, "%s: rows of %s overlap one another", what,
                name);
  return KVD_OK;
}

// Whether any vector of r (d wide) has bytes in [p, p + bytes). Vectors are
// gone through only where the span of all of them meets that range.
bool rows_meet(const kvd_rows *r, int d, const void *p, size_t bytes) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(r->data);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p), hi = lo + bytes;
  const auto meet = [&](uintptr_t at, int64_t last) {  // to element last + d
    return at < hi && at + 2 * (uintptr_t)(last + d) > lo;
  };
  const int64_t rs = r->row_stride, hs = r->head_stride;
  const int64_t heads = (r->heads - 1) * hs;
  if (!meet(base, (r->rows - 1) * rs + heads)) return false;
  for (int32_t i = 0; i < r->rows; ++i) {
    const uintptr_t row = base + 2 * (uintptr_t)(i * rs);
    if (!meet(row, heads)) continue;
    for (int32_t h = 0; h < r->heads; ++h)
      if (meet(row + 2 * (uintptr_t)(h * hs), 0)) return true;
  }
  return false;
}

bool rows_aligned16(const kvd_rows *r) {
  return aligned(r->data, 16) && r->row_stride % 8 == 0 &&
         r->head_stride % 8 == 0;
}

// A rotation's input and output pair.
kvd_status check_rotated(const kvd_rows *in, const kvd_rows *out, int d,
                         const char *what, const char *name) {
  if (!in || !out)
    return fail(KVD_ERR_NULL, "%s: %s and %s_out go together", what, name,
                name);
  kvd_status st = check_rows(in, d, false, what, name);
  if (st != KVD_OK) return st;
  st = check_rows(out, d, true, what, name);
  if (st != KVD_OK) return st;
  if (in->rows != out->rows || in->heads != out->heads)
    return fail(KVD_ERR_SHAPE, "%s: %s and %s_out have different shapes", what,
                name, name);
  if (in->rows > 0 && in->data == out->data &&
      (in->row_stride != out->row_stride ||
       in->head_stride != out->head_stride))
    return fail(KVD_ERR_SHAPE, "%s: %s_out in place needs the strides of %s",
                what, name, name);
  return KVD_OK;
}

kvd_status check_rope(const kvd_rope_plan *r, const int32_t *positions,
                      int64_t axis_stride, int d, int rows,
                      const char *what) {
  if (r->d_rot < 2 || r->d_rot % 2 != 0 || r->d_rot > d)
    return fail(KVD_ERR_SHAPE, "%s: d_rot (%d) must be even, at least 2 and "
                "at most the head width %d", what, r->d_rot, d);
  if (r->d_rot > 1024 || r->n_axes < 1 || r->n_axes > 4)
    return fail(KVD_ERR_UNSUPPORTED, "%s: d_rot up to 1024 and 1 to 4 axes",
                what);
  if (r->pairing != KVD_PAIR_HALF && r->pairing != KVD_PAIR_ADJACENT)
    return fail(KVD_ERR_UNSUPPORTED, "%s: unknown pairing %d", what,
                r->pairing);
  if (r->inverse != 0 && r->inverse != 1)
    return fail(KVD_ERR_SHAPE, "%s: inverse must be 0 or 1", what);
  if (!r->turns || (rows > 0 && !positions))
    return fail(KVD_ERR_NULL, "%s: turns and positions required", what);
  if (!aligned(r->turns, 8) || !aligned(positions, 4))
    return fail(KVD_ERR_SHAPE, "%s: turns or positions misaligned", what);
  if (r->n_axes > 1 && axis_stride < rows)
    return fail(KVD_ERR_SHAPE, "%s: axis_stride below the number of rows",
                what);
  return KVD_OK;
}

void set_rope(kvd::RowsParams &p, const kvd_rope_plan *r,
              const int32_t *positions, int64_t axis_stride) {
  p.rope.turns = r->turns;
  p.rope.axis = r->axis;
  p.rope.pos = positions;
  p.rope.axis_stride = axis_stride;
  p.rope.half = r->d_rot / 2;
  p.rope.n_axes = r->n_axes;
  p.rope.adjacent = r->pairing == KVD_PAIR_ADJACENT;
  p.rope.inverse = r->inverse;
  p.rope.on = 1;
}

void set_q(kvd::RowsParams &p, const kvd_rows *q, const kvd_rows *q_out) {
  p.q = static_cast<const uint16_t *>(q->data);
  p.q_rs = q->row_stride;
  p.q_hs = q->head_stride;
  p.q_out = static_cast<uint16_t *>(q_out->data);
  p.qo_rs = q_out->row_stride;
  p.qo_hs = q_out->head_stride;
  p.n_h = q->heads;
}

// What kvd_kv_write and kvd_kv_read check alike.
kvd_status check_paged_rows(const kvd_cache *c, int32_t max_blocks,
                            const int32_t *block_table, const int32_t *start,
                            const int32_t *row_start, int32_t batch,
                            const char *what) {
  if (batch < 0 || batch > 65535 || max_blocks < 1)
    return fail(KVD_ERR_SHAPE, "%s: 0 <= batch <= 65535 and "
                "max_blocks_per_seq >= 1 required", what);
  if (c->head_dim % 8 != 0)
    return fail(KVD_ERR_SHAPE, "%s: head_dim must be a multiple of 8", what);
  if (batch > 0 && (!block_table || !start || !row_start))
    return fail(KVD_ERR_NULL, "%s: block_table, start and row_start required",
                what);
  return KVD_OK;
}

kvd_status check_kv_rows(const kvd_cache *c, const kvd_rows *r, int rows,
                         bool out, const char *what, const char *name) {
  const kvd_status st = check_rows(r, c->head_dim, out, what, name);
  if (st != KVD_OK) return st;
  if (r->heads != c->n_kv || r->rows != rows)
    return fail(KVD_ERR_SHAPE, "%s: %s must have %d rows of %d heads", what,
                name, rows, c->n_kv);
  if (!rows_aligned16(r))
    return fail(KVD_ERR_SHAPE, "%s: %s must be 16-byte aligned with strides "
                "that are multiples of 8", what, name);
  return KVD_OK;
}

void set_paged(kvd::RowsParams &p, const kvd_cache *c, int32_t max_blocks,
               const int32_t *block_table, const int32_t *start,
               const int32_t *row_start, int32_t batch, int *err) {
  p.k_cache = static_cast<uint8_t *>(c->k);
  p.v_cache = static_cast<uint8_t *>(c->v);
  p.k_inv = c->k_inv_scale;
  p.v_inv = c->v_inv_scale;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.block_table = block_table;
  p.start = start;
  p.row_start = row_start;
  p.n_kv = c->n_kv;
  p.d = c->head_dim;
  p.dtype = c->dtype;
  p.batch = batch;
  p.max_blocks = max_blocks;
  p.block_size = c->block_size;
  p.num_blocks = c->num_blocks;
  p.err = err;
}

struct ExtendPlan {
  bool few = false;
  kvd::FewPlan f{};
  kvd::ExtendParams p{};  // n_splits, whole_units, chunks_per_split
  int blocks = 0, splits = 1;
  size_t ws_o_bytes = 0, ws_bytes = 0;
};

// Few (row, head) pairs a kv head (at most 16): the stream-K kernel with one
// CTA per SM. Else blocks of 256 pairs a CTA, or of 512 a pair of CTAs where
// a sequence may have more than 256 (one prompt chunk of 1,021 tokens over
// 32,000, 56 heads: 698 us with pairs, 792 without). Blocks that make two waves
// and more are not split over the positions. Of several sequences, fewer are
// split into 8 / 7 waves of parts, were all as long as max_seq_len: ragged
// ones then fill about one, and blocks that already make 8 / 7 waves are left
// whole. (Means over eight draws of lengths, us, for 16 sequences of 4 rows to
// 16K positions, 6 of 9 to 8K, 4 of 175 to 12K, 3 of 30 to 32K: 105, 36, 198,
// 99; one wave 115, 39, 198, 101; two waves 106, 46, 209, 109; three 106, 46,
// 221, 115. Equally long sequences of 1.2 to 1.5 waves would gain up to 9% from
// two or three parts: 4 of 200 rows over 12,000 positions 369 and 356, 3 of 250
// over 16,000 474 and 435.) One sequence's blocks are about equally long, and
// the number of parts whose last wave ends first is taken (the chunk above: 3
// waves of halves, 722 us when thirds, in 4.4 waves, took 802). A choice by the
// lengths themselves, on the device, cost every CTA 1 to 4 us.
ExtendPlan extend_plan(const kvd_cache *c, const kvd_seqs *s, int rows,
                       int max_rows, int n_h, int sms) {
  ExtendPlan pl;
  const int g = n_h / c->n_kv;
  const int forced = g_decode_ctas.load(std::memory_order_relaxed);
  if ((long)max_rows * g <= kvd::kFewPairs) {
    pl.few = true;
    const kvd::FewPlan f =
        kvd::extend_few_plan(c->n_kv, c->block_size, max_rows * g, s->batch,
                             s->max_seq_len, sms);
    pl.f = f;
    const long units = (long)s->batch * (c->n_kv / f.hp);
    long unit_chunks = ((long)s->max_seq_len + f.chunk - 1) / f.chunk;
    const long chunks = units * unit_chunks;
    if (s->window > 0)
      unit_chunks = std::min<long>(
          unit_chunks,
          ((long)s->window + max_rows + f.chunk - 2) / f.chunk + 1);
    long ctas = forced > 0 ? forced : sms;
    if (forced <= 0 && units <= ctas &&
        unit_chunks * f.chunk <= kWholeUnitChunks * kvd::kStageRows) {
      pl.p.whole_units = 1;
      pl.p.n_splits = (int)std::max(units, 1L);
      return pl;
    }
    ctas = std::max(1L, std::min(ctas, std::max(chunks, 1L)));
    pl.p.n_splits = (int)ctas;
    if (chunks >= 8 * ctas) pl.p.gap = kvd::kUnitGap;
    const size_t slots = (size_t)ctas * 2 * f.hp * 8 * f.tiles;
    pl.ws_o_bytes = round_up(slots * 128 * 4, 256);
    pl.ws_bytes = pl.ws_o_bytes + round_up(slots * 4, 256);
    return pl;
  }
  const long pairs = (long)rows * g;
  const int ctas_per_block = (long)max_rows * g > kvd::kExtendRows ? 2 : 1;
  const int block_rows = ctas_per_block * kvd::kExtendRows;
  pl.p.block_rows = block_rows;
  pl.blocks =
      (int)((pairs + (long)std::min(s->batch, rows) * (block_rows - 1)) /
            block_rows);
  const int ch = kvd::kExtendChunk;
  long chunks = ((long)s->max_seq_len + ch - 1) / ch;
  if (s->window > 0)
    chunks = std::min<long>(
        chunks, ((long)s->window + block_rows / g + ch) / ch + 2);
  const long ctas = (long)pl.blocks * c->n_kv * ctas_per_block;
  const long want = forced > 0 ? forced : 8L * sms / 7;
  if (forced > 0 || ctas < 2L * sms) {
    long per = (ctas * chunks + want - 1) / want;
    if (forced <= 0 && s->batch == 1) {
      // a part costs kPartCost chunks beyond its own: its queries, the
      // filling and emptying of the pipeline, its share of the merge
      constexpr long kPartCost = 4;
      long best = -1;
      for (long w = 1; w <= 16; ++w) {  // waves, and the parts that fill them
        const long n = std::min(w * sms / ctas, chunks);
        if (n < 1) continue;
        const long each = (chunks + n - 1) / n;
        const long cost =
            (ctas * n + sms - 1) / sms * (each + kPartCost);
        if (best < 0 || cost < best) best = cost, per = each;
      }
    }
    // (a launch has at most 65,535 splits)
    per = std::max({4L, per, (chunks + 65534) / 65535});
    if (per < chunks) {
      pl.p.chunks_per_split = (int)per;
      pl.splits = (int)((chunks + per - 1) / per);
      const size_t n = (size_t)pl.splits * rows * n_h;
      pl.ws_o_bytes = round_up(n * 128 * 4, 256);
      pl.ws_bytes = pl.ws_o_bytes + round_up(n * 4, 256);
    }
  }
  return pl;
}

kvd_status check_extend(const kvd_cache *c, const kvd_seqs *s, int rows,
                        int max_rows, int n_h, bool lists,
                        const char *what) {
  kvd_status st = check_cache(c, true, what);
  if (st != KVD_OK) return st;
  st = check_seqs(s, c, what);
  if (st != KVD_OK) return st;
  if (c->dtype != KVD_MXFP4)
    return fail(KVD_ERR_UNSUPPORTED, "%s: an MXFP4 cache is required", what);
  if (n_h < 1 || n_h % c->n_kv != 0)
    return fail(KVD_ERR_SHAPE, "%s: n_h (%d) must be a positive multiple of "
                "n_kv (%d)", what, n_h, c->n_kv);
  if (n_h / c->n_kv > 128)
    return fail(KVD_ERR_UNSUPPORTED, "%s: group size %d above 128", what,
                n_h / c->n_kv);
  if (s->batch > 1024)
    return fail(KVD_ERR_UNSUPPORTED, "%s: at most 1024 sequences per call "
                "(got %d)", what, s->batch);
  if (rows < 0 || max_rows < 0)
    return fail(KVD_ERR_SHAPE, "%s: rows and max_rows must be >= 0", what);
  if (!lists && (rows != s->batch || max_rows != 1))
    return fail(KVD_ERR_SHAPE, "%s: without row_start there is one row a "
                "sequence (rows = batch, max_rows = 1)", what);
  if ((long)rows * n_h >= (1L << 31) || (long)max_rows * n_h >= (1L << 31))
    return fail(KVD_ERR_SHAPE, "%s: rows x n_h must be below 2^31", what);
  return KVD_OK;
}

}  // namespace

extern "C" {

kvd_status kvd_rope_turns(const double *freq, int32_t n, uint64_t *turns) {
  if (n < 0) return fail(KVD_ERR_SHAPE, "rope_turns: n must be >= 0");
  if (n > 0 && (!freq || !turns))
    return fail(KVD_ERR_NULL, "rope_turns: freq and turns required");
  for (int32_t i = 0; i < n; ++i)
    if (!(std::fabs(freq[i]) < 2147483648.0))
      return fail(KVD_ERR_SHAPE, "rope_turns: frequency %d is not finite and "
                  "below 2^31 in magnitude", i);
  // 1 / (2 pi) as the sum of two doubles
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int32_t i = 0; i < n; ++i) {
    const double f = std::fabs(freq[i]);
    const double a = f * hi;  // a + b turns
    const double b = std::fma(f, lo, std::fma(f, hi, -a));
    // fractions of a turn in units of 2^-64, modulo 2^64
    const double t = std::ldexp(a - std::floor(a), 32);  // exact
    const double r = std::ldexp(t - std::floor(t), 32) + std::ldexp(b, 64);
    const uint64_t u = ((uint64_t)std::floor(t) << 32) +
                       (uint64_t)(int64_t)std::nearbyint(r);
    turns[i] = freq[i] < 0 ? 0 - u : u;
  }
  return ok();
}

kvd_status kvd_rope(const kvd_rope_plan *plan, const int32_t *positions,
                    int64_t axis_stride, int32_t head_dim, const kvd_rows *q,
                    const kvd_rows *q_out, const kvd_rows *k,
                    const kvd_rows *k_out, kvd_stream stream) {
  if (!plan) return fail(KVD_ERR_NULL, "rope: plan is NULL");
  if (head_dim < 1) return fail(KVD_ERR_SHAPE, "rope: head_dim must be >= 1");
  kvd_status st = check_rotated(q, q_out, head_dim, "rope", "q");
  if (st != KVD_OK) return st;
  if (k || k_out) {
    st = check_rotated(k, k_out, head_dim, "rope", "k");
    if (st != KVD_OK) return st;
    if (k->rows != q->rows)
      return fail(KVD_ERR_SHAPE, "rope: q and k have different rows");
  }
  st = check_rope(plan, positions, axis_stride, head_dim, q->rows, "rope");
  if (st != KVD_OK) return st;
  if (q->rows == 0) return ok();
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  kvd::RowsParams p{};
  set_rope(p, plan, positions, axis_stride);
  set_q(p, q, q_out);
  if (k) {
    p.k = static_cast<const uint16_t *>(k->data);
    p.k_rs = k->row_stride;
    p.k_hs = k->head_stride;
    p.k_out = static_cast<uint16_t *>(k_out->data);
    p.ko_rs = k_out->row_stride;
    p.ko_hs = k_out->head_stride;
    p.n_kv = k->heads;
  }
  p.rows = q->rows;
  p.d = head_dim;
  p.err = d->err;
  return launched(kvd::launch_rows(p, false, d->sms,
                                   reinterpret_cast<cudaStream_t>(stream)),
                  "rope");
}

kvd_status kvd_kv_write(const kvd_cache *cache, const int32_t *block_table,
                        int32_t max_blocks_per_seq, const int32_t *start,
                        const int32_t *row_start, int32_t batch,
                        const kvd_rows *k_new, const kvd_rows *v_new,
                        const kvd_rope_plan *rope, const int32_t *positions,
                        int64_t axis_stride, const kvd_rows *q,
                        const kvd_rows *q_out, kvd_stream stream) {
  kvd_status st = check_cache(cache, false, "kv_write");
  if (st != KVD_OK) return st;
  st = check_paged_rows(cache, max_blocks_per_seq, block_table, start,
                        row_start, batch, "kv_write");
  if (st != KVD_OK) return st;
  if (!k_new) return fail(KVD_ERR_NULL, "kv_write: k_new required");
  if (cache->v && !v_new)
    return fail(KVD_ERR_NULL, "kv_write: v_new required for a K/V cache");
  st = check_kv_rows(cache, k_new, k_new->rows, false, "kv_write", "k_new");
  if (st != KVD_OK) return st;
  if (cache->v) {
    st = check_kv_rows(cache, v_new, k_new->rows, false, "kv_write", "v_new");
    if (st != KVD_OK) return st;
  }
  if (cache->dtype == KVD_FP8_E4M3 &&
      (!cache->k_inv_scale || (cache->v && !cache->v_inv_scale)))
    return fail(KVD_ERR_NULL, "kv_write: fp8 cache needs inverse scales");
  if (q || q_out) {
    if (!rope)
      return fail(KVD_ERR_NULL, "kv_write: q is rotated, so rope is required");
    st = check_rotated(q, q_out, cache->head_dim, "kv_write", "q");
    if (st != KVD_OK) return st;
    if (q->rows != k_new->rows)
      return fail(KVD_ERR_SHAPE, "kv_write: q and k_new have different rows");
  }
  if (rope) {
    st = check_rope(rope, positions, axis_stride, cache->head_dim, k_new->rows,
                    "kv_write");
    if (st != KVD_OK) return st;
    if (!kvd::rows_fit(cache->head_dim, rope->d_rot / 2))
      return fail(KVD_ERR_UNSUPPORTED, "kv_write: a rotated head of %d does "
                  "not fit in shared memory", cache->head_dim);
  }
  if (batch == 0 || k_new->rows == 0) return ok();
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  kvd::RowsParams p{};
  set_paged(p, cache, max_blocks_per_seq, block_table, start, row_start, batch,
            d->err);
  p.k = static_cast<const uint16_t *>(k_new->data);
  p.k_rs = k_new->row_stride;
  p.k_hs = k_new->head_stride;
  if (cache->v) {
    p.v = static_cast<const uint16_t *>(v_new->data);
    p.v_rs = v_new->row_stride;
    p.v_hs = v_new->head_stride;
  }
  if (rope) set_rope(p, rope, positions, axis_stride);
  if (q) set_q(p, q, q_out);
  p.rows = k_new->rows;
  return launched(kvd::launch_rows(p, true, d->sms,
                                   reinterpret_cast<cudaStream_t>(stream)),
                  "kv_write");
}

kvd_status kvd_kv_read(const kvd_cache *cache, const int32_t *block_table,
                       int32_t max_blocks_per_seq, const int32_t *start,
                       const int32_t *row_start, int32_t batch,
                       const kvd_rows *k_out, const kvd_rows *v_out,
                       kvd_stream stream) {
  kvd_status st = check_cache(cache, v_out != nullptr, "kv_read");
  if (st != KVD_OK) return st;
  st = check_paged_rows(cache, max_blocks_per_seq, block_table, start,
                        row_start, batch, "kv_read");
  if (st != KVD_OK) return st;
  if (!k_out && !v_out)
    return fail(KVD_ERR_NULL, "kv_read: k_out or v_out required");
  const int rows = k_out ? k_out->rows : v_out->rows;
  if (k_out) {
    st = check_kv_rows(cache, k_out, rows, true, "kv_read", "k_out");
    if (st != KVD_OK) return st;
  }
  if (v_out) {
    st = check_kv_rows(cache, v_out, rows, true, "kv_read", "v_out");
    if (st != KVD_OK) return st;
  }
  if (cache->dtype == KVD_FP8_E4M3 &&
      ((k_out && !cache->k_scale) || (v_out && !cache->v_scale)))
    return fail(KVD_ERR_NULL, "kv_read: fp8 cache needs scales");
  if (batch == 0 || rows == 0) return ok();
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  kvd::RowsParams p{};
  set_paged(p, cache, max_blocks_per_seq, block_table, start, row_start, batch,
            d->err);
  if (k_out) {
    p.k_out = static_cast<uint16_t *>(k_out->data);
    p.ko_rs = k_out->row_stride;
    p.ko_hs = k_out->head_stride;
  }
  if (v_out) {
    p.v_out = static_cast<uint16_t *>(v_out->data);
    p.vo_rs = v_out->row_stride;
    p.vo_hs = v_out->head_stride;
  }
  p.rows = rows;
  return launched(kvd::launch_read(p, d->sms,
                                   reinterpret_cast<cudaStream_t>(stream)),
                  "kv_read");
}

kvd_status kvd_extend_workspace_size(const kvd_cache *cache,
                                     const kvd_seqs *seqs, int32_t rows,
                                     int32_t max_rows, int32_t n_h,
                                     size_t *bytes) {
  if (!bytes)
    return fail(KVD_ERR_NULL, "extend_workspace_size: bytes is NULL");
  kvd_status st = check_extend(cache, seqs, rows, max_rows, n_h, true,
                               "extend_workspace_size");
  if (st != KVD_OK) return st;
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  *bytes = rows == 0 || max_rows == 0 || seqs->batch == 0
               ? 0
               : extend_plan(cache, seqs, rows, max_rows, n_h, d->sms)
                     .ws_bytes;
  return ok();
}

kvd_status kvd_gqa_extend(const kvd_cache *cache, const kvd_seqs *seqs,
                          const int32_t *row_start, int32_t max_rows,
                          const kvd_rows *q, float scale, void *out,
                          float *lse, void *workspace, size_t workspace_bytes,
                          kvd_stream stream) {
  if (!q) return fail(KVD_ERR_NULL, "gqa_extend: q is NULL");
  kvd_status st = check_extend(cache, seqs, q->rows, max_rows, q->heads,
                               row_start != nullptr, "gqa_extend");
  if (st != KVD_OK) return st;
  st = check_rows(q, cache->head_dim, false, "gqa_extend", "q");
  if (st != KVD_OK) return st;
  if (!rows_aligned16(q) || !aligned(out, 16))
    return fail(KVD_ERR_SHAPE, "gqa_extend: q and out must be 16-byte aligned, "
                "q's strides multiples of 8");
  if (seqs->batch == 0 || q->rows == 0 || max_rows == 0) return ok();
  if (!out) return fail(KVD_ERR_NULL, "gqa_extend: out required");
  if (rows_meet(q, cache->head_dim, out,
                (size_t)q->rows * q->heads * cache->head_dim * 2))
    return fail(KVD_ERR_SHAPE, "gqa_extend: out overlaps q");
  const DeviceInfo *d = nullptr;
  st = device_info(&d);
  if (st != KVD_OK) return st;
  const int n_h = q->heads;
  const ExtendPlan pl =
      extend_plan(cache, seqs, q->rows, max_rows, n_h, d->sms);
  Plan need;
  need.ws_bytes = pl.ws_bytes;
  st = check_ws(need, workspace, workspace_bytes, "gqa_extend");
  if (st != KVD_OK) return st;
  kvd::ExtendParams p = pl.p;
  p.k = static_cast<const uint8_t *>(cache->k);
  p.v = static_cast<const uint8_t *>(cache->v);
  p.block_table = seqs->block_table;
  p.seq_lens = seqs->seq_lens;
  p.q = static_cast<const uint16_t *>(q->data);
  p.q_rs = q->row_stride;
  p.q_hs = q->head_stride;
  p.out = static_cast<uint16_t *>(out);
  p.lse = lse;
  p.ws_o = static_cast<float *>(workspace);
  p.ws_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                       pl.ws_o_bytes);
  p.batch = seqs->batch;
  p.n_h = n_h;
  p.n_kv = cache->n_kv;
  p.dk = p.dv = cache->head_dim;
  p.dtype = cache->dtype;
  p.block_size = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.max_blocks = seqs->max_blocks_per_seq;
  p.max_seq_len = seqs->max_seq_len;
  p.window = seqs->window;
  p.win_start = seqs->window_start;
  p.row_start = row_start;
  p.max_rows = max_rows;
  p.rows = q->rows;
  p.scale_log2 = log2_scale(scale, cache->head_dim);
  p.err = d->err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return launched(pl.few
                      ? kvd::launch_extend_few(p, pl.f, s)
                      : kvd::launch_extend_tc(p, pl.blocks, pl.splits, s),
                  "gqa_extend");
}

}  // extern "C"
