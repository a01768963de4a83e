// mbk_kv4_api.cu -- the C entry points of the 4-bit KV cache's operators (include/mbk.h): argument
// checks and launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/mbk.h"
#include "mbk_kv4.h"

using namespace mbk;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Makes `device` current for the scope and puts the caller's back.
struct DeviceScope {
  int before = -1, device;
  bool ok;
  explicit DeviceScope(int d) : device(d) {
    ok = cudaGetDevice(&before) == cudaSuccess && (before == d || cudaSetDevice(d) == cudaSuccess);
  }
  ~DeviceScope() {
    if (before >= 0 && before != device) cudaSetDevice(before);
  }
};

// SMs of a device; 0 for one that does not exist or is not the architecture this library is built for.
int sms_of(int device) {
  static std::atomic<int> known[64];
  if (device < 0 || device >= 64) return 0;
  int n = known[device].load(std::memory_order_relaxed);
  if (n != 0) return n;
  int major = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess || major != 10 ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return 0;
  known[device].store(n, std::memory_order_relaxed);
  return n;
}

bool batch_ok(const mbk_kv4_config& c, const mbk_kv4_batch* b) {
  if (!b || b->n_seq < 1 || b->n_seq > MBK_KV4_MAX_SEQS || b->n_tokens < 1 || b->max_count < 1 || b->max_count > b->n_tokens ||
      b->max_rows < 0 || (int64_t)b->max_rows > (int64_t)c.max_pages * c.page_size || !b->offsets || !b->rows || !b->tables ||
      (b->positions && !c.track))
    return false;
  return aligned4(b->offsets) && aligned4(b->rows) && aligned4(b->positions) && aligned4(b->tables) && aligned4(b->status);
}

bool rows_ok(const void* p, int64_t ld, int64_t least, int32_t dtype) {
  const int64_t unit = dtype == MBK_KV4_BF16 ? 8 : 4;
  return p && aligned16(p) && ld >= least && ld % unit == 0;
}

Kv4Batch batch_of(const mbk_kv4_batch& b) {
  return Kv4Batch{b.n_seq, b.n_tokens, b.max_count, b.max_rows, b.offsets, b.rows, b.positions, b.tables, b.status};
}

int launched(cudaError_t e) { return e == cudaSuccess ? MBK_OK : MBK_ERR_CUDA; }

bool common_ok(const mbk_kv4_config* cfg, const void* pool, int32_t layer, int32_t dtype) {
  return kv4_config_check(cfg) == MBK_OK && pool && aligned16(pool) && layer >= 0 && layer < cfg->n_layers &&
         (dtype == MBK_KV4_FP32 || dtype == MBK_KV4_BF16);
}

}  // namespace

extern "C" {

int64_t mbk_kv4_pool_bytes(const mbk_kv4_config* cfg) {
  if (kv4_config_check(cfg) != MBK_OK) return MBK_ERR_INVALID_ARG;
  const Kv4Geom g = kv4_geom(*cfg, nullptr);
  if ((double)g.page_stride * cfg->num_pages > 9e18) return MBK_ERR_INVALID_ARG;
  return (int64_t)(g.page_stride * (unsigned long long)cfg->num_pages);
}

int mbk_kv4_append(const mbk_kv4_config* cfg, void* pool, int32_t layer, const mbk_kv4_batch* batch, const void* k, const void* v,
                   int64_t ld, int32_t dtype, void* stream) {
  if (!common_ok(cfg, pool, layer, dtype) || !batch_ok(*cfg, batch)) return MBK_ERR_INVALID_ARG;
  const int64_t row = (int64_t)cfg->n_kv_heads * cfg->head_dim;
  if (!rows_ok(k, ld, row, dtype) || !rows_ok(v, ld, row, dtype)) return MBK_ERR_INVALID_ARG;
  if (sms_of(cfg->device) == 0) return MBK_ERR_UNSUPPORTED;
  DeviceScope d(cfg->device);
  if (!d.ok) return MBK_ERR_CUDA;
  return launched(kv4_append(kv4_geom(*cfg, pool), layer, batch_of(*batch), k, v, ld, dtype == MBK_KV4_BF16, (cudaStream_t)stream));
}

int mbk_kv4_read(const mbk_kv4_config* cfg, const void* pool, int32_t layer, const mbk_kv4_batch* batch, void* k, void* v, int64_t ld,
                 int32_t dtype, void* stream) {
  if (!common_ok(cfg, pool, layer, dtype) || !batch_ok(*cfg, batch)) return MBK_ERR_INVALID_ARG;
  const int64_t row = (int64_t)cfg->n_kv_heads * cfg->head_dim;
  if (!rows_ok(k, ld, row, dtype) || !rows_ok(v, ld, row, dtype)) return MBK_ERR_INVALID_ARG;
  if (sms_of(cfg->device) == 0) return MBK_ERR_UNSUPPORTED;
  DeviceScope d(cfg->device);
  if (!d.ok) return MBK_ERR_CUDA;
  return launched(
      kv4_read(kv4_geom(*cfg, const_cast<void*>(pool)), layer, batch_of(*batch), k, v, ld, dtype == MBK_KV4_BF16, (cudaStream_t)stream));
}

int64_t mbk_kv4_attention_workspace(const mbk_kv4_config* cfg, const mbk_kv4_batch* batch) {
  if (kv4_config_check(cfg) != MBK_OK || !batch || batch->n_seq < 1 || batch->n_seq > MBK_KV4_MAX_SEQS || batch->n_tokens < 1 ||
      batch->max_count < 1 || batch->max_count > batch->n_tokens || batch->max_rows < 0 ||
      (int64_t)batch->max_rows > (int64_t)cfg->max_pages * cfg->page_size)
    return MBK_ERR_INVALID_ARG;
  const int sms = sms_of(cfg->device);
  if (sms == 0) return MBK_ERR_UNSUPPORTED;
  return (int64_t)kv4_attention_workspace(kv4_geom(*cfg, nullptr), batch_of(*batch), sms);
}

int mbk_kv4_attention(const mbk_kv4_config* cfg, void* pool, int32_t layer, const mbk_kv4_batch* batch, const void* q, int64_t ldq,
                      void* out, int64_t ldo, int32_t dtype, float scale, float cap, const float* slopes, int32_t window,
                      int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!common_ok(cfg, pool, layer, dtype) || !batch_ok(*cfg, batch)) return MBK_ERR_INVALID_ARG;
  const int64_t row = (int64_t)cfg->n_heads * cfg->head_dim;
  if (!rows_ok(q, ldq, row, dtype) || !rows_ok(out, ldo, row, dtype) || q == out || !std::isfinite(scale) ||
      !(cap >= 0.f) || !std::isfinite(cap) || !aligned4(slopes) || window < 0 || (accumulate != 0 && accumulate != 1) ||
      (accumulate && !cfg->track))
    return MBK_ERR_INVALID_ARG;
  // the split counts blocks of rows in 32 bits, tiles of 8 query rows at least
  const double tiles = std::ceil((double)batch->max_count * (cfg->n_heads / cfg->n_kv_heads) / 8.0);
  if (tiles * batch->n_seq * cfg->n_kv_heads * (batch->max_rows / 32 + 1) > 2e9 || tiles > (1 << 24)) return MBK_ERR_INVALID_ARG;
  const int sms = sms_of(cfg->device);
  if (sms == 0) return MBK_ERR_UNSUPPORTED;
  const Kv4Geom g = kv4_geom(*cfg, pool);
  const Kv4Batch b = batch_of(*batch);
  const int64_t need = (int64_t)kv4_attention_workspace(g, b, sms);
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return MBK_ERR_INVALID_ARG;
  DeviceScope d(cfg->device);
  if (!d.ok) return MBK_ERR_CUDA;
  const Kv4Attn a{q, out, ldq, ldo, dtype == MBK_KV4_BF16, scale, cap, slopes, window, accumulate};
  return launched(kv4_attention(g, layer, b, a, workspace, sms, (cudaStream_t)stream));
}

int64_t mbk_kv4_evict_workspace(const mbk_kv4_config* cfg, int32_t n_layers, int32_t n_seq, int32_t keep) {
  if (kv4_config_check(cfg) != MBK_OK || n_layers < 1 || n_layers > cfg->n_layers || n_seq < 1 || n_seq > MBK_KV4_MAX_SEQS || keep < 1 ||
      (int64_t)keep > (int64_t)cfg->max_pages * cfg->page_size)
    return MBK_ERR_INVALID_ARG;
  return (int64_t)kv4_evict_workspace(kv4_geom(*cfg, nullptr), n_layers, n_seq, keep);
}

int mbk_kv4_evict(const mbk_kv4_config* cfg, void* pool, int32_t layer, int32_t n_layers, int32_t n_seq, int32_t max_rows,
                  const int32_t* rows, const int32_t* tables, const int32_t* next_pos, int32_t keep, int32_t recent,
                  const int32_t* out_tables, int32_t out_pages, int32_t* rows_out, int32_t* status, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  if (!common_ok(cfg, pool, layer, MBK_KV4_FP32) || !cfg->track || n_layers < 1 || n_layers > cfg->n_layers - layer || n_seq < 1 ||
      n_seq > MBK_KV4_MAX_SEQS || max_rows < 1 || max_rows > MBK_KV4_MAX_EVICT_ROWS ||
      (int64_t)max_rows > (int64_t)cfg->max_pages * cfg->page_size || !rows || !tables || !next_pos || !rows_out || keep < 1 || (int64_t)keep > (int64_t)cfg->max_pages * cfg->page_size || recent < 0 || recent > keep)
    return MBK_ERR_INVALID_ARG;
  if (!aligned4(rows) || !aligned4(tables) || !aligned4(next_pos) || !aligned4(out_tables) || !aligned4(rows_out) || !aligned4(status))
    return MBK_ERR_INVALID_ARG;
  if (out_tables && (out_pages < 1 || (int64_t)std::min(keep, max_rows) > (int64_t)out_pages * cfg->page_size)) return MBK_ERR_INVALID_ARG;
  const double segs = (double)n_layers * n_seq * cfg->n_kv_heads;
  if (segs * (std::min(keep, max_rows) / 32 + 1) > 2e9) return MBK_ERR_INVALID_ARG;
  const Kv4Geom g = kv4_geom(*cfg, pool);
  if (!workspace || !aligned16(workspace) || workspace_bytes < (int64_t)kv4_evict_workspace(g, n_layers, n_seq, keep))
    return MBK_ERR_INVALID_ARG;
  const int sms = sms_of(cfg->device);
  if (sms == 0) return MBK_ERR_UNSUPPORTED;
  DeviceScope d(cfg->device);
  if (!d.ok) return MBK_ERR_CUDA;
  return launched(kv4_evict(g, layer, n_layers, n_seq, max_rows, rows, tables, next_pos, keep, recent, out_tables, out_pages, rows_out,
                            status, workspace, sms, (cudaStream_t)stream));
}

}  // extern "C"
