// mbk_kv4_rows.cu -- the 4-bit KV cache's rows: append (quantise), read, and eviction by accumulated
// attention weight.  Also the pool's geometry.
#include "mbk_kv4_device.h"

namespace mbk {
namespace {

// ------------------------------------------------------------------ append and read
// Eight lanes hold a group of 64, 8 elements each; a block of threads takes `per` tokens of one
// sequence (grid.y).  Bound by the bytes: 8 n d elements read, 0.56 bytes written for each.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// code = (x - lo) / scale to nearest even, in 0 .. 15.  The product with 1 / scale is within 2^-22 of
// the quotient's 15 at most, so only a product nearer than 1e-5 to a half needs the division itself
// (bf16 inputs do meet exact halves).
__device__ __forceinline__ uint32_t code_of(float x, float lo, float scale, float inv) {
  const float t = __fsub_rn(x, lo);
  float q = __fmul_rn(t, inv);
  const float h = q - floorf(q) - 0.5f;
  if (fabsf(h) < 1e-5f) q = __fdiv_rn(t, scale);
  return (uint32_t)fminf(fmaxf(rintf(q), 0.f), 15.f);
}

template <typename T, int D>
__global__ void __launch_bounds__(256) append_kernel(Kv4Geom g, int layer, Kv4Batch b, const T* k, const T* v, long long ld, int per) {
  const int s = blockIdx.y;
  const SeqView q = seq_view(g, b, s, threadIdx.x == 0 && blockIdx.x == 0);
  const int t0 = blockIdx.x * per;
  if (t0 >= q.c) return;
  if (q.r < q.c) {
    if (threadIdx.x == 0) flag(b.status, MBK_KV4_BAD_BATCH);
    return;
  }
  const int nt = min(per, q.c - t0);
  const int32_t* table = b.tables + (size_t)s * g.max_pages;
  constexpr int V = D / 8;  // vectors of 8 in a row
  const int work = nt * g.nkv * 2 * V;
  const int p0 = b.positions != nullptr ? b.positions[s] : q.r - q.c;
  for (int e = threadIdx.x; e < (work + 31) / 32 * 32; e += blockDim.x) {
    const bool on = e < work;  // groups of 8 lanes are all on or all off
    const int ee = on ? e : 0;
    const int j = ee % V, hv = ee / V, sel = hv & 1, th = hv >> 1, h = th % g.nkv, t = t0 + th / g.nkv;
    float x[8];
    load8<T>((sel ? v : k) + (size_t)(q.tok0 + t) * ld + h * D + 8 * j, x);
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = x[i] != x[i] ? x[i] : fminf(fmaxf(x[i], -65504.f), 65504.f);
      lo = min_nan(lo, x[i]);
      hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, m));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)), lh = __float2half_rn(lo);
    const float sf = __half2float(sh), lf = __half2float(lh);
    uint32_t w = 0;
    if (sf > 0.f) {  // a constant group, and one with a NaN, has codes of zero
      const float inv = __fdiv_rn(1.f, sf);
#pragma unroll
      for (int i = 0; i < 8; ++i) w |= code_of(x[i], lf, sf, inv) << (4 * i);
    }
    if (!on) continue;
    const int row = q.r - q.c + t, lane_row = row % kRows;
    uint8_t* blk = block_of(g, table, layer, h, row, b.status);
    if (blk == nullptr) continue;
    uint8_t* base = blk + sel * half_bytes(D);
    *reinterpret_cast<uint32_t*>(base + lane_row * (D / 2) + 4 * j) = w;
    if (j % 8 == 0) {
      const __half2 p = __halves2half2(sh, lh);
      *reinterpret_cast<__half2*>(base + code_bytes(D) + (lane_row * (D / 64) + j / 8) * 4) = p;
    }
    if (g.track && sel == 0 && j == 0) {
      *reinterpret_cast<int32_t*>(blk + pos_at(D) + 4 * lane_row) = p0 + t;
      *reinterpret_cast<float*>(blk + weight_at(D) + 4 * lane_row) = 0.f;
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) read_kernel(Kv4Geom g, int layer, Kv4Batch b, T* k, T* v, long long ld, int per) {
  const int s = blockIdx.y;
  const SeqView q = seq_view(g, b, s, threadIdx.x == 0 && blockIdx.x == 0);
  const int t0 = blockIdx.x * per;
  if (t0 >= q.c) return;
  if (q.r < q.c) {
    if (threadIdx.x == 0) flag(b.status, MBK_KV4_BAD_BATCH);
    return;
  }
  const int nt = min(per, q.c - t0);
  const int32_t* table = b.tables + (size_t)s * g.max_pages;
  constexpr int V = D / 8;
  const int work = nt * g.nkv * 2 * V;
  for (int e = threadIdx.x; e < work; e += blockDim.x) {
    const int j = e % V, hv = e / V, sel = hv & 1, th = hv >> 1, h = th % g.nkv, t = t0 + th / g.nkv;
    const int row = q.r - q.c + t, lane_row = row % kRows;
    const uint8_t* blk = block_of(g, table, layer, h, row, b.status);
    float x[8];
    if (blk == nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
    } else {
      const uint8_t* base = blk + sel * half_bytes(D);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(base + lane_row * (D / 2) + 4 * j);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(base + code_bytes(D) + (lane_row * (D / 64) + j / 8) * 4));
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(p.x, (float)((w >> (4 * i)) & 15u), p.y);
    }
    store8((sel ? v : k) + (size_t)(q.tok0 + t) * ld + h * D + 8 * j, x);
  }
}

// ------------------------------------------------------------------ eviction
// select_kernel, one CTA per (layer, sequence, KV head): the keep-th largest key by radix selection
// (keys: the order of the weights, the recent rows above all), equal keys lowest row first; then the
// map: dest row j < keep takes row map[j] -- itself if it is kept, else the next kept row from above.
constexpr int kSelThreads = 1024;
constexpr int kKeysInSmem = 40960;

__device__ __forceinline__ uint32_t weight_key(float w, int pos, int young) {
  if (pos >= young) return 0xffffffffu;
  if (w != w) w = 0.f;  // NaN counts as no weight
  w += 0.f;             // -0 as +0
  const uint32_t u = __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct EvictArgs {
  Kv4Geom g;
  int layer0, n_layers, n_seq, max_rows, keep, recent, out_pages;
  const int32_t *rows, *tables, *next_pos, *out_tables;
  int32_t *rows_out, *status;
  int32_t* map;     // [segment][keep]
  int32_t* movers;  // [segment][keep]
  int32_t* kept;    // [segment] rows that are left
};

__device__ int block_sum_scan(int v, int* sums, int* total) {  // exclusive scan over the block; all threads call
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int t = sums[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, t, m);
      if (lane >= m) t += y;
    }
    sums[lane] = t;
  }
  __syncthreads();
  *total = sums[31];
  return x - v + (warp > 0 ? sums[warp - 1] : 0);
}

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int hist[2048];
  __shared__ int sums[32];
  __shared__ int s_bin, s_above;
  const int seg = blockIdx.x, h = seg % a.g.nkv, s = seg / a.g.nkv % a.n_seq, layer = a.layer0 + seg / (a.g.nkv * a.n_seq);
  const int tid = threadIdx.x;
  int r = a.rows[s];
  if (r < 0 || r > a.max_rows) {
    if (tid == 0) flag(a.status, MBK_KV4_BAD_BATCH);
    r = min(max(r, 0), a.max_rows);
  }
  const int keep = a.keep;
  int32_t* map = a.map + (size_t)seg * keep;
  if (tid == 0) a.kept[seg] = min(r, keep);
  if (r <= keep) {
    for (int i = tid; i < r; i += kSelThreads) map[i] = i;
    return;
  }
  const int32_t* table = a.tables + (size_t)s * a.g.max_pages;
  const int young = a.next_pos[s] - a.recent;
  const int words = (r + 31) / 32;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);                 // kept rows
  uint32_t* keys = bits + (a.max_rows + 31) / 32;                     // [r] when they fit
  const bool cached = a.max_rows <= kKeysInSmem;
  auto load_key = [&](int row) -> uint32_t {
    const uint8_t* p = block_of(a.g, table, layer, h, row, a.status);
    if (p == nullptr) return 0u;
    return weight_key(*reinterpret_cast<const float*>(p + weight_at(D) + 4 * (row % kRows)),
                      *reinterpret_cast<const int*>(p + pos_at(D) + 4 * (row % kRows)), young);
  };
  if (cached)
    for (int i = tid; i < r; i += kSelThreads) keys[i] = load_key(i);
  auto key = [&](int row) { return cached ? keys[row] : load_key(row); };
  // digits of 11, 11 and 10 bits from the top
  uint32_t prefix = 0, mask = 0;
  int need = keep;  // rows still to be taken from those that share the prefix
  const int shift[3] = {21, 10, 0}, width[3] = {2048, 2048, 1024};
  for (int pass = 0; pass < 3; ++pass) {
    for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < r; i += kSelThreads) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift[pass]) & (width[pass] - 1)], 1);
    }
    __syncthreads();
    // thread t holds bins from the top: 2047 - 2 t and 2046 - 2 t
    const int b0 = 2047 - 2 * tid, h0 = hist[b0], h1 = hist[b0 - 1];
    int total;
    const int above = block_sum_scan(h0 + h1, sums, &total);
    if (above < need && above + h0 >= need) {
      s_bin = b0;
      s_above = above;
    } else if (above + h0 < need && above + h0 + h1 >= need) {
      s_bin = b0 - 1;
      s_above = above + h0;
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift[pass];
    mask |= (uint32_t)(width[pass] - 1) << shift[pass];
    need -= s_above;
    __syncthreads();
  }
  // rows above the threshold, and the first `need` rows equal to it
  int taken = 0;
  for (int i0 = 0; i0 < r; i0 += kSelThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < r ? key(i) : 0u;
    const bool eq = i < r && k == prefix;
    int total;
    const int before = taken + block_sum_scan(eq ? 1 : 0, sums, &total);
    const bool take = i < r && (k > prefix || (eq && before < need));
    const uint32_t b = __ballot_sync(0xffffffffu, take);
    if ((tid & 31) == 0 && i / 32 < words) bits[i / 32] = b;
    taken += total;
  }
  __syncthreads();
  // kept rows from `keep` on, in order
  int32_t* movers = a.movers + (size_t)seg * keep;
  int done = 0;
  for (int w0 = keep / 32; w0 < words; w0 += kSelThreads) {
    const int w = w0 + tid;
    uint32_t b = w < words ? bits[w] : 0u;
    if (w == keep / 32) b &= ~0u << (keep % 32);
    int total;
    int at = done + block_sum_scan(__popc(b), sums, &total);
    for (; b != 0u; b &= b - 1) movers[at++] = w * 32 + __ffs(b) - 1;
    done += total;
  }
  __syncthreads();
  done = 0;
  const int kw = (keep + 31) / 32;
  for (int w0 = 0; w0 < kw; w0 += kSelThreads) {
    const int w = w0 + tid;
    uint32_t b = 0u, in = 0u;
    if (w < kw) {
      in = w == keep / 32 ? (1u << (keep % 32)) - 1u : ~0u;
      b = ~bits[w] & in;
    }
    int total;
    int at = done + block_sum_scan(__popc(b), sums, &total);
    if (w < kw)
      for (int i = 0; i < 32; ++i)
        if (in >> i & 1u) map[w * 32 + i] = (b >> i & 1u) ? movers[at++] : w * 32 + i;
    done += total;
  }
}

// move_kernel: 32 destination rows of a segment per CTA.  In place (no out_tables) a kept row below
// `keep` stays and the others come from rows >= keep, so no row is both read and written.
template <int D>
__global__ void __launch_bounds__(256) move_kernel(const __grid_constant__ EvictArgs a) {
  const int nb = (min(a.keep, a.max_rows) + kRows - 1) / kRows, seg = blockIdx.x / nb, rb = blockIdx.x - seg * nb;
  const int h = seg % a.g.nkv, s = seg / a.g.nkv % a.n_seq, layer = a.layer0 + seg / (a.g.nkv * a.n_seq);
  const int n = a.kept[seg], r0 = rb * kRows;
  if (rb == 0 && h == 0 && layer == a.layer0 && threadIdx.x == 0) a.rows_out[s] = n;
  if (r0 >= n) return;
  const bool in_place = a.out_tables == nullptr;
  const int32_t* table = a.tables + (size_t)s * a.g.max_pages;
  const int32_t* to = in_place ? table : a.out_tables + (size_t)s * a.out_pages;
  const int32_t* map = a.map + (size_t)seg * a.keep;
  uint8_t* dst = block_of(a.g, to, layer, h, r0, threadIdx.x == 0 ? a.status : nullptr);
  if (dst == nullptr) return;
  constexpr int C = D / 32;  // 16-byte chunks of a row's codes
  const int rows = min(kRows, n - r0);
  for (int i = threadIdx.x; i < rows * 2 * (C + 1); i += blockDim.x) {
    const int row = i / (2 * (C + 1)), part = i % (2 * (C + 1)), sel = part / (C + 1), c = part % (C + 1);
    const int src = map[r0 + row];
    if (in_place && src == r0 + row) continue;
    const uint8_t* from = block_of(a.g, table, layer, h, src, a.status);
    if (from == nullptr) continue;
    const int fr = src % kRows;
    const uint8_t* f = from + sel * half_bytes(D);
    uint8_t* d = dst + sel * half_bytes(D);
    if (c < C) {
      *reinterpret_cast<uint4*>(d + row * (D / 2) + 16 * c) = *reinterpret_cast<const uint4*>(f + fr * (D / 2) + 16 * c);
    } else {
#pragma unroll
      for (int g = 0; g < D / 64; ++g)
        reinterpret_cast<uint32_t*>(d + code_bytes(D))[row * (D / 64) + g] = reinterpret_cast<const uint32_t*>(f + code_bytes(D))[fr * (D / 64) + g];
      const int at = sel ? weight_at(D) : pos_at(D);
      reinterpret_cast<uint32_t*>(dst + at)[row] = reinterpret_cast<const uint32_t*>(from + at)[fr];
    }
  }
}

// Tokens of a CTA of append and read: about 2,048 vectors of 8.
int tokens_per_cta(const Kv4Geom& g) { return std::max(1, 2048 / (g.nkv * 2 * (g.d / 8))); }

constexpr int kSelectSmem = 208 * 1024;  // dynamic shared memory of the selection: 227 KB less its static part

}  // namespace

size_t kv4_evict_workspace(const Kv4Geom& g, int n_layers, int n_seq, int keep) {
  const size_t segs = (size_t)n_layers * n_seq * g.nkv;
  return 2 * round256(segs * keep * 4) + round256(segs * 4);
}

cudaError_t kv4_append(const Kv4Geom& g, int layer, const Kv4Batch& b, const void* k, const void* v, long long ld, int bf16,
                       cudaStream_t st) {
  const int per = tokens_per_cta(g);
  const dim3 grid((unsigned)((b.max_count + per - 1) / per), (unsigned)b.n_seq);
  if (bf16) {
    const auto *kk = (const __nv_bfloat16*)k, *vv = (const __nv_bfloat16*)v;
    return g.d == 64 ? launch(append_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per)
                     : launch(append_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per);
  }
  const auto *kk = (const float*)k, *vv = (const float*)v;
  return g.d == 64 ? launch(append_kernel<float, 64>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per)
                   : launch(append_kernel<float, 128>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per);
}

cudaError_t kv4_read(const Kv4Geom& g, int layer, const Kv4Batch& b, void* k, void* v, long long ld, int bf16, cudaStream_t st) {
  const int per = tokens_per_cta(g);
  const dim3 grid((unsigned)((b.max_count + per - 1) / per), (unsigned)b.n_seq);
  if (bf16) {
    auto *kk = (__nv_bfloat16*)k, *vv = (__nv_bfloat16*)v;
    return g.d == 64 ? launch(read_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per)
                     : launch(read_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per);
  }
  auto *kk = (float*)k, *vv = (float*)v;
  return g.d == 64 ? launch(read_kernel<float, 64>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per)
                   : launch(read_kernel<float, 128>, grid, 256, 0, st, false, g, layer, b, kk, vv, ld, per);
}

cudaError_t kv4_evict(const Kv4Geom& g, int layer0, int n_layers, int n_seq, int max_rows, const int32_t* rows,
                      const int32_t* tables, const int32_t* next_pos, int keep, int recent, const int32_t* out_tables,
                      int out_pages, int32_t* rows_out, int32_t* status, void* ws, cudaStream_t st) {
  static std::atomic<bool> once[2][64];
  const size_t segs = (size_t)n_layers * n_seq * g.nkv;
  EvictArgs a;
  a.g = g;
  a.layer0 = layer0;
  a.n_layers = n_layers;
  a.n_seq = n_seq;
  a.max_rows = max_rows;
  a.keep = keep;
  a.recent = recent;
  a.out_pages = out_pages;
  a.rows = rows;
  a.tables = tables;
  a.next_pos = next_pos;
  a.out_tables = out_tables;
  a.rows_out = rows_out;
  a.status = status;
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  a.map = reinterpret_cast<int32_t*>(w);
  a.movers = reinterpret_cast<int32_t*>(w + round256(segs * keep * 4));
  a.kept = reinterpret_cast<int32_t*>(w + 2 * round256(segs * keep * 4));
  const size_t smem = (size_t)(max_rows + 31) / 32 * 4 + (max_rows <= kKeysInSmem ? (size_t)max_rows * 4 : 0);
  if (cudaError_t e = allow_smem(g.d == 64 ? (const void*)select_kernel<64> : (const void*)select_kernel<128>, once[g.d == 128], kSelectSmem)) return e;
  const dim3 mg((unsigned)((std::min(keep, max_rows) + kRows - 1) / kRows * segs));
  if (g.d == 64) {
    if (cudaError_t e = launch(select_kernel<64>, dim3((unsigned)segs), kSelThreads, smem, st, false, a)) return e;
    return launch(move_kernel<64>, mg, 256, 0, st, false, a);
  }
  if (cudaError_t e = launch(select_kernel<128>, dim3((unsigned)segs), kSelThreads, smem, st, false, a)) return e;
  return launch(move_kernel<128>, mg, 256, 0, st, false, a);
}

int kv4_config_check(const mbk_kv4_config* c) {
  if (!c || c->device < 0 || c->n_layers < 1 || c->n_heads < 1 || c->n_kv_heads < 1 || c->n_heads % c->n_kv_heads != 0 ||
      c->n_heads / c->n_kv_heads > kKv4MaxGroup || c->n_heads > 65535 || (c->head_dim != 64 && c->head_dim != 128) || c->num_pages < 1 ||
      c->max_pages < 1 || c->page_size < kKv4Rows || c->page_size > (1 << 20) || (c->page_size & (c->page_size - 1)) != 0 ||
      (c->track != 0 && c->track != 1))
    return MBK_ERR_INVALID_ARG;
  if ((long long)c->max_pages * c->page_size > 1 << 27) return MBK_ERR_INVALID_ARG;
  const long long block = kKv4Rows * (c->head_dim + c->head_dim / 64 * 8 + (c->track ? 8 : 0));
  if (block * (c->page_size / kKv4Rows) > 0x7fffffffll) return MBK_ERR_INVALID_ARG;
  return MBK_OK;
}

Kv4Geom kv4_geom(const mbk_kv4_config& c, void* pool) {
  Kv4Geom g;
  g.pool = reinterpret_cast<uint8_t*>(pool);
  g.num_pages = c.num_pages;
  g.L = c.n_layers;
  g.nq = c.n_heads;
  g.nkv = c.n_kv_heads;
  g.d = c.head_dim;
  g.track = c.track;
  g.page_shift = 0;
  while ((1 << g.page_shift) < c.page_size) ++g.page_shift;
  g.max_pages = c.max_pages;
  g.block_bytes = kKv4Rows * (c.head_dim + c.head_dim / 64 * 8 + (c.track ? 8 : 0));
  g.head_stride = (unsigned)(g.block_bytes * (c.page_size / kKv4Rows));
  g.page_stride = (unsigned long long)c.n_layers * c.n_kv_heads * g.head_stride;
  return g;
}

}  // namespace mbk
