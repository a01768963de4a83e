// mbk_kv4_rows.cu -- the 4-bit KV cache's rows: append (quantise), read, and eviction by accumulated
// attention weight.  Also the pool's geometry.
#include <climits>

#include "mbk_kv4_device.h"

namespace mbk {
namespace {

// ------------------------------------------------------------------ append and read
// A row -- the K or V of one token and KV head -- is d / 16 lanes of 16 elements.  A CTA takes `per` tokens of one
// sequence (grid.y).  Both are bound by instructions rather than bytes unless those for an element are few: 16
// elements share a row's address, there is no division by the number of heads (a multiplication by its
// reciprocal), codes go through the low bits of a large float or half instead of conversions (one in four
// clocks), and arithmetic goes two values at a time.  Measured: append of 16 ragged prompts of up to 1,000 tokens, 8 KV heads,
// d 128, bf16: 20 us a launch (2.3 TB/s; issue slots 74% busy); read of 24 sequences of 2,048 rows, 32 KV heads, d 64, to
// bf16: 516 MB in 88 us, 5.9 TB/s (87% of a copy's rate).
struct RowsArgs {
  Kv4Geom g;
  Kv4Batch b;
  int layer, per;
  unsigned by_heads;  // ceil(2^32 / nkv), 0 for one head
  long long ld;
};
struct RowAt {
  int t, h, sel;
};
__device__ __forceinline__ RowAt row_at(const RowsArgs& a, int r) {  // r < 2 nkv per
  const unsigned th = (unsigned)r >> 1;
  const int t = a.by_heads == 0u ? (int)th : (int)__umulhi(th, a.by_heads);
  return RowAt{t, (int)th - t * a.g.nkv, r & 1};
}

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

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The codes of 8 elements: (x - lo) / scale to nearest even, in 0 .. 15.  The product with 1 / scale is within 2^-22
// of the quotient's 15 at most, so only where one lies nearer than 1e-5 to a half the divisions themselves are made
// (bf16 inputs do meet exact halves).  Adding 1.5 * 2^23 rounds to nearest even and leaves the code in the low bits; the
// words add up with the big number's own bits, which are taken off at the end.
__device__ __forceinline__ uint32_t codes_of(const float* x, float lo, float scale, float inv) {
  constexpr float kBig = 12582912.f;
  constexpr uint32_t kBits = 0x4b400000u, kExtra = kBits * 0x11111111u;  // kBits << 0, 4, .. 28 added up
  const f2 less = pair_of(-lo, -lo), by = pair_of(inv, inv), big = pair_of(kBig, kBig), no_big = pair_of(-kBig, -kBig), minus = pair_of(-1.f, -1.f);
  float far = 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float2 q = halves(mul2(sum2(pair_of(x[i], x[i + 1]), less), by));
    q.x = fminf(fmaxf(q.x, 0.f), 15.f);
    q.y = fminf(fmaxf(q.y, 0.f), 15.f);
    const f2 c = pair_of(q.x, q.y), r = sum2(c, big);
    const float2 d = halves(fma2(sum2(r, no_big), minus, c)), rr = halves(r);
    far = fmaxf(far, fmaxf(fabsf(d.x), fabsf(d.y)));
    w += __float_as_uint(rr.x) * (1u << (4 * i)) + __float_as_uint(rr.y) * (1u << (4 * i + 4));
  }
  w -= kExtra;
  if (far > 0.49999f) {
    w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[i], lo), scale)), 0.f), 15.f) << (4 * i);
  }
  return w;
}

template <typename T, int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ RowsArgs a, const T* k, const T* v) {
  constexpr int V = D / 16, kStep = 256 / V;  // lanes of a row, rows of a step
  const Kv4Geom& g = a.g;
  const int s = blockIdx.y, t0 = blockIdx.x * a.per;
  const SeqView q = seq_view(g, a.b, s, threadIdx.x == 0 && blockIdx.x == 0);
  if (t0 >= q.c) return;
  if (q.r < q.c) {
    if (threadIdx.x == 0) flag(a.b.status, MBK_KV4_BAD_BATCH);
    return;
  }
  const int rows = min(a.per, q.c - t0) * g.nkv * 2, j = threadIdx.x % V, first = threadIdx.x / V;
  const int32_t* table = a.b.tables + (size_t)s * g.max_pages;
  const int p0 = a.b.positions != nullptr ? a.b.positions[s] : q.r - q.c;
  for (int r0 = 0; r0 < rows; r0 += kStep) {  // all lanes of a warp go round together
    const bool on = r0 + first < rows;
    RowAt at = row_at(a, on ? r0 + first : 0);
    at.t += t0;
    const T* from = (at.sel ? v : k) + (size_t)(q.tok0 + at.t) * a.ld + at.h * D + 16 * j;
    float x[16];
    load8<T>(from, *reinterpret_cast<float(*)[8]>(&x[0]));
    load8<T>(from + 8, *reinterpret_cast<float(*)[8]>(&x[8]));
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 15; i += 2) {
      lo = min3_nan(lo, x[i], x[i + 1]);
      hi = max3_nan(hi, x[i], x[i + 1]);
    }
    lo = min_nan(lo, x[15]);
    hi = max_nan(hi, x[15]);
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, m));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    if (!(lo >= -65504.f && hi <= 65504.f)) {  // beyond fp16, or NaN, which stays
      lo = lo != lo ? lo : fminf(fmaxf(lo, -65504.f), 65504.f);
      hi = hi != hi ? hi : fminf(fmaxf(hi, -65504.f), 65504.f);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = fminf(fmaxf(x[i], -65504.f), 65504.f);
    }
    const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)), lh = __float2half_rn(lo);
    const float sf = __half2float(sh), lf = __half2float(lh);
    uint2 w = make_uint2(0u, 0u);  // a constant group, and one with a NaN, has codes of zero
    if (sf > 0.f) {
      const float inv = __fdiv_rn(1.f, sf);
      w.x = codes_of(x, lf, sf, inv);
      w.y = codes_of(x + 8, lf, sf, inv);
    }
    if (on) {
      const int row = q.r - q.c + at.t, lane_row = row % kRows;
      uint8_t* blk = block_of(g, table, a.layer, at.h, row, a.b.status);
      if (blk != nullptr) {
        uint8_t* base = blk + at.sel * half_bytes(D);
        *reinterpret_cast<uint2*>(base + lane_row * (D / 2) + 8 * j) = w;
        if (j % 4 == 0)
          *reinterpret_cast<__half2*>(base + code_bytes(D) + (lane_row * (D / 64) + j / 4) * 4) = __halves2half2(sh, lh);
        if (g.track && at.sel == 0 && j == 0) {
          *reinterpret_cast<int32_t*>(blk + pos_at(D) + 4 * lane_row) = p0 + at.t;
          *reinterpret_cast<float*>(blk + weight_at(D) + 4 * lane_row) = 0.f;
        }
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256) read_kernel(const __grid_constant__ RowsArgs a, T* k, T* v) {
  constexpr int V = D / 16, kStep = 256 / V, kAtOnce = 2;
  const Kv4Geom& g = a.g;
  const int s = blockIdx.y, t0 = blockIdx.x * a.per;
  const SeqView q = seq_view(g, a.b, s, threadIdx.x == 0 && blockIdx.x == 0);
  if (t0 >= q.c) return;
  if (q.r < q.c) {
    if (threadIdx.x == 0) flag(a.b.status, MBK_KV4_BAD_BATCH);
    return;
  }
  const int rows = min(a.per, q.c - t0) * g.nkv * 2, j = threadIdx.x % V, first = threadIdx.x / V;
  const int32_t* table = a.b.tables + (size_t)s * g.max_pages;
  // a lane's 16 elements are 8 of each half of the row, so that neighbouring lanes write neighbouring bytes
  for (int r0 = 0; r0 < rows; r0 += kAtOnce * kStep) {
    uint32_t w[kAtOnce][2], pr[kAtOnce][2];
    T* to[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int r = r0 + u * kStep + first;
      to[u] = nullptr;
      if (r < rows) {
        RowAt at = row_at(a, r);
        at.t += t0;
        const int row = q.r - q.c + at.t, lane_row = row % kRows;
        const uint8_t* blk = block_of(g, table, a.layer, at.h, row, a.b.status);
        const uint8_t* base = blk + at.sel * half_bytes(D);
        to[u] = (at.sel ? v : k) + (size_t)(q.tok0 + at.t) * a.ld + at.h * D + 8 * j;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          w[u][hf] = pr[u][hf] = 0u;  // a bad page reads as zero
          if (blk != nullptr) {
            w[u][hf] = __ldg(reinterpret_cast<const uint32_t*>(base + lane_row * (D / 2) + hf * (D / 4) + 4 * j));
            pr[u][hf] = __ldg(reinterpret_cast<const uint32_t*>(base + code_bytes(D) + (lane_row * (D / 64) + hf * (D / 128)) * 4));
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (to[u] == nullptr) continue;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float2 p = unpack_half(pr[u][hf]);
        const f2 scale = pair_of(p.x, p.x), lo = pair_of(p.y, p.y);
        const uint32_t word = w[u][hf];
        float x[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // codes i and i + 4 as 1024 + code in fp16
          const uint32_t c = (word >> (4 * i) & 0x000f000fu) | 0x64006400u;
          const float2 f = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&c), __float2half2_rn(1024.f)));
          const float2 y = halves(fma2(pair_of(f.x, f.y), scale, lo));
          x[i] = y.x;
          x[i + 4] = y.y;
        }
        store8(to[u] + hf * (D / 2), x);
      }
    }
  }
}

// ------------------------------------------------------------------ eviction
// select_kernel, one CTA per (layer, sequence, KV head): the keep-th largest key by radix selection (keys: the order
// of the weights, the recent rows above all), equal keys lowest row first; then the map: dest row j < keep takes row
// map[j] -- itself if it is kept, else the next kept row from above.  Bound by its chain of passes and barriers
// rather than by bytes (20 MB read in 45 us for 512 segments of up to 8,192 rows, 0.44 TB/s).
constexpr int kKeysInSmem = 32768;

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
  int32_t* kept;    // [segment] rows that are left, or -1: the sequence's row count is out of bounds
};

template <int NT>
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
  int t = lane < NT / 32 ? sums[lane] : 0;  // every warp scans the warps' sums for itself
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, t, m);
    if (lane >= m) t += y;
  }
  *total = __shfl_sync(0xffffffffu, t, 31);
  return x - v + (warp > 0 ? __shfl_sync(0xffffffffu, t, warp - 1) : 0);
}

template <int D, int NT>
__global__ void __launch_bounds__(NT) select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int hist[2048];
  __shared__ int sums[32];
  __shared__ int s_bin, s_above, s_in;
  const int seg = blockIdx.x, h = seg % a.g.nkv, s = seg / a.g.nkv % a.n_seq, layer = a.layer0 + seg / (a.g.nkv * a.n_seq);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = a.rows[s];
  const bool bad = r < 0 || r > a.max_rows;  // left as it is
  const int keep = a.keep;
  int32_t* map = a.map + (size_t)seg * keep;
  if (tid == 0) {
    if (bad) flag(a.status, MBK_KV4_BAD_BATCH);
    a.kept[seg] = bad ? -1 : min(r, keep);
  }
  if (bad) return;
  if (r <= keep) {
    for (int i = tid; i < r; i += NT) map[i] = i;
    return;
  }
  const int32_t* table = a.tables + (size_t)s * a.g.max_pages;
  const int young = max(a.next_pos[s], INT_MIN + a.recent) - a.recent;
  const int words = (r + 31) / 32, all_words = (a.max_rows + 31) / 32;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);             // kept rows
  int* ranks = reinterpret_cast<int*>(bits + all_words);          // [all_words + 1] free rows (kept rows from `keep` on) before a word
  uint32_t* keys = reinterpret_cast<uint32_t*>(ranks + all_words + 1);  // [r] when they fit
  const bool cached = a.max_rows <= kKeysInSmem;
  auto load_key = [&](int row) -> uint32_t {
    const uint8_t* p = block_of(a.g, table, layer, h, row, a.status);
    if (p == nullptr) return 0u;
    return weight_key(__ldg(reinterpret_cast<const float*>(p + weight_at(D) + 4 * (row % kRows))),
                      __ldg(reinterpret_cast<const int*>(p + pos_at(D) + 4 * (row % kRows))), young);
  };
  if (cached) {
    for (int i0 = tid; i0 < r; i0 += 4 * NT) {
      uint32_t k[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) k[u] = i0 + u * NT < r ? load_key(i0 + u * NT) : 0u;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i0 + u * NT < r) keys[i0 + u * NT] = k[u];
    }
  }
  auto key = [&](int row) { return cached ? keys[row] : load_key(row); };
  // digits of 11, 11 and 10 bits from the top
  uint32_t prefix = 0, mask = 0;
  int need = keep;  // rows still to be taken from those that share the prefix
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, width = pass == 2 ? 1024 : 2048;
    for (int i = tid; i < 2048; i += NT) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < r; i += NT) {
      const uint32_t k = key(i);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (width - 1)], 1);
    }
    __syncthreads();
    // thread t holds kBins bins from the top: 2047 - kBins t and below
    constexpr int kBins = 2048 / NT;
    int n[kBins], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins; ++i) sum += n[i] = hist[2047 - kBins * tid - i];
    int total;
    int above = block_sum_scan<NT>(sum, sums, &total);
#pragma unroll
    for (int i = 0; i < kBins; ++i) {
      if (above < need && above + n[i] >= need) {
        s_bin = 2047 - kBins * tid - i;
        s_above = above;
        s_in = n[i];
      }
      above += n[i];
    }
    __syncthreads();
    prefix |= (uint32_t)s_bin << shift;
    mask |= (uint32_t)(width - 1) << shift;
    need -= s_above;
    if (s_in == need) {  // all that share the prefix are taken: nothing more to tell apart (a key of 0 ends this too)
      if (prefix != 0u) {
        prefix -= 1u;
        need = 0;
        break;
      }
    }
  }
  // Rows above the threshold, and the first `need` rows equal to it.  Each warp has a run of whole words of rows, so that
  // one scan over the warps' counts is enough.
  const int per = (words + NT / 32 - 1) / (NT / 32), w_from = min(words, warp * per), w_to = min(words, w_from + per);
  int before = 0;
  if (need > 0) {
    int equal = 0, all;
    for (int w = w_from; w < w_to; ++w) {
      const int i = w * 32 + lane;
      equal += __popc(__ballot_sync(0xffffffffu, i < r && key(i) == prefix));
    }
    before = block_sum_scan<NT>(lane == 0 ? equal : 0, sums, &all);
    before = __shfl_sync(0xffffffffu, before, 0);
  }
  // and in the same walk the free rows below `keep` (the kept ones above) before each word, from the warp's first on
  int free_rows = 0, moved = 0;
  for (int w = w_from; w < w_to; ++w) {
    const int i = w * 32 + lane;
    const uint32_t k = i < r ? key(i) : 0u;
    const uint32_t eq = __ballot_sync(0xffffffffu, i < r && k == prefix);
    const bool mine = (eq >> lane & 1u) && before + __popc(eq & ((1u << lane) - 1u)) < need;
    const uint32_t b = __ballot_sync(0xffffffffu, mine || (i < r && k > prefix));
    before += __popc(eq);
    const uint32_t below = w < keep / 32 ? ~0u : w == keep / 32 ? (1u << (keep % 32)) - 1u : 0u;  // rows < keep of the word
    if (lane == 0) {
      bits[w] = b;
      if (below != 0u) ranks[w] = free_rows;       // words up to keep / 32
      if (below != ~0u) ranks[w + 1] = moved;      // words from keep / 32 on, one place further
    }
    free_rows += __popc(~b & below);
    moved += __popc(b & ~below);
  }
  int total;
  const int free_base = __shfl_sync(0xffffffffu, block_sum_scan<NT>(lane == 0 ? free_rows : 0, sums, &total), 0);
  const int moved_base = __shfl_sync(0xffffffffu, block_sum_scan<NT>(lane == 0 ? moved : 0, sums, &total), 0);
  for (int w = w_from + lane; w < w_to; w += 32) {
    if (w * 32 < keep) ranks[w] += free_base;
    if (w >= keep / 32) ranks[w + 1] += moved_base;
  }
  __syncthreads();
  int32_t* movers = a.movers + (size_t)seg * keep;  // kept rows from `keep` on, in order
  for (int i = keep + tid; i < r; i += NT) {
    const uint32_t b = bits[i / 32] & (i / 32 == keep / 32 ? ~0u << (keep % 32) : ~0u);
    if (b >> (i % 32) & 1u) movers[ranks[i / 32 + 1] + __popc(b & ((1u << (i % 32)) - 1u))] = i;
  }
  __syncthreads();
  for (int j = tid; j < keep; j += NT) {
    const uint32_t free_bits = ~bits[j / 32];
    map[j] = free_bits >> (j % 32) & 1u ? movers[ranks[j / 32] + __popc(free_bits & ((1u << (j % 32)) - 1u))] : j;
  }
}

// move_kernel: kMove destination rows of a segment per CTA.  First where each row comes from (map, page table), then
// the bytes, 16 at a time, several copies under way per thread: 63 us for 512 segments of 2,048 rows at d 128, 318 MB, 5.0
// TB/s (75% of a copy's rate; rows are 64 bytes of codes and four words in six places).  In place (no out_tables) a kept row below `keep`
// stays and the others come from rows >= keep, so no row is both read and written.
constexpr int kMove = 128;
template <int D>
__global__ void __launch_bounds__(256) move_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ const uint8_t* from[kMove];  // block of the source row, or null: nothing to move
  __shared__ uint8_t* to[kMove];
  __shared__ unsigned char lane_of[kMove];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nb = (min(a.keep, a.max_rows) + kMove - 1) / kMove, seg = blockIdx.x / nb, rb = blockIdx.x - seg * nb;
  const int h = seg % a.g.nkv, s = seg / a.g.nkv % a.n_seq, layer = a.layer0 + seg / (a.g.nkv * a.n_seq);
  const int n = a.kept[seg], r0 = rb * kMove;
  if (rb == 0 && h == 0 && layer == a.layer0 && threadIdx.x == 0) a.rows_out[s] = n < 0 ? a.rows[s] : n;
  if (r0 >= n) return;
  const int rows = min(kMove, n - r0);
  if (threadIdx.x < rows) {
    const bool in_place = a.out_tables == nullptr;
    const int32_t* table = a.tables + (size_t)s * a.g.max_pages;
    const int32_t* out = in_place ? table : a.out_tables + (size_t)s * a.out_pages;
    const int row = r0 + threadIdx.x, src = a.map[(size_t)seg * a.keep + row];
    const uint8_t* f = in_place && src == row ? nullptr : block_of(a.g, table, layer, h, src, a.status);
    uint8_t* d = f == nullptr ? nullptr : block_of(a.g, out, layer, h, row, a.status);
    from[threadIdx.x] = d == nullptr ? nullptr : f;
    to[threadIdx.x] = d;
    lane_of[threadIdx.x] = (unsigned char)(src % kRows);
  }
  __syncthreads();
  constexpr int C = D / 32, kAtOnce = 4;  // 16-byte chunks of a row's codes
  // codes: rows x (K, V) x C chunks
  for (int i0 = threadIdx.x; i0 < rows * 2 * C; i0 += 256 * kAtOnce) {
    uint4 x[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + 256 * u, row = i / (2 * C), sel = i / C % 2, c = i % C;
      if (i < rows * 2 * C && from[row] != nullptr)
        x[u] = __ldg(reinterpret_cast<const uint4*>(from[row] + sel * half_bytes(D) + lane_of[row] * (D / 2) + 16 * c));
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + 256 * u, row = i / (2 * C), sel = i / C % 2, c = i % C;
      if (i < rows * 2 * C && from[row] != nullptr)
        *reinterpret_cast<uint4*>(to[row] + sel * half_bytes(D) + (r0 + row) % kRows * (D / 2) + 16 * c) = x[u];
    }
  }
  // pairs of K and V, position, weight: 4 bytes each
  constexpr int G = D / 64, P = 2 * G + 2;
  for (int i0 = threadIdx.x; i0 < rows * P; i0 += 256 * kAtOnce) {
    uint32_t x[kAtOnce];
    auto place = [&](int part, int lane) {  // byte of part `part` of row `lane` in its block
      return part < 2 * G ? part / G * half_bytes(D) + code_bytes(D) + (lane * G + part % G) * 4
                          : (part == 2 * G ? pos_at(D) : weight_at(D)) + 4 * lane;
    };
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + 256 * u, row = i / P;
      if (i < rows * P && from[row] != nullptr) x[u] = *reinterpret_cast<const uint32_t*>(from[row] + place(i % P, lane_of[row]));
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + 256 * u, row = i / P;
      if (i < rows * P && from[row] != nullptr) *reinterpret_cast<uint32_t*>(to[row] + place(i % P, (r0 + row) % kRows)) = x[u];
    }
  }
}

// Tokens of a CTA of append and read: about 1,024 vectors of 16.
int tokens_per_cta(const Kv4Geom& g) { return std::max(1, 1024 / (g.nkv * 2 * (g.d / 16))); }

constexpr int kSelectSmem = 208 * 1024;  // dynamic shared memory of the selection: 227 KB less its static part

}  // namespace

size_t kv4_evict_workspace(const Kv4Geom& g, int n_layers, int n_seq, int keep) {
  const size_t segs = (size_t)n_layers * n_seq * g.nkv;
  return 2 * round256(segs * keep * 4) + round256(segs * 4);
}

namespace {
RowsArgs rows_args(const Kv4Geom& g, int layer, const Kv4Batch& b, long long ld) {
  RowsArgs a;
  a.g = g;
  a.b = b;
  a.layer = layer;
  a.per = tokens_per_cta(g);
  a.by_heads = g.nkv == 1 ? 0u : (unsigned)(((1ull << 32) + g.nkv - 1) / g.nkv);
  a.ld = ld;
  return a;
}
dim3 rows_grid(const RowsArgs& a) { return dim3((unsigned)((a.b.max_count + a.per - 1) / a.per), (unsigned)a.b.n_seq); }
}  // namespace

cudaError_t kv4_append(const Kv4Geom& g, int layer, const Kv4Batch& b, const void* k, const void* v, long long ld, int bf16,
                       cudaStream_t st) {
  const RowsArgs a = rows_args(g, layer, b, ld);
  const dim3 grid = rows_grid(a);
  if (bf16) {
    const auto *kk = (const __nv_bfloat16*)k, *vv = (const __nv_bfloat16*)v;
    return g.d == 64 ? launch(append_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, false, a, kk, vv)
                     : launch(append_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, false, a, kk, vv);
  }
  const auto *kk = (const float*)k, *vv = (const float*)v;
  return g.d == 64 ? launch(append_kernel<float, 64>, grid, 256, 0, st, false, a, kk, vv)
                   : launch(append_kernel<float, 128>, grid, 256, 0, st, false, a, kk, vv);
}

cudaError_t kv4_read(const Kv4Geom& g, int layer, const Kv4Batch& b, void* k, void* v, long long ld, int bf16, cudaStream_t st) {
  const RowsArgs a = rows_args(g, layer, b, ld);
  const dim3 grid = rows_grid(a);
  if (bf16) {
    auto *kk = (__nv_bfloat16*)k, *vv = (__nv_bfloat16*)v;
    return g.d == 64 ? launch(read_kernel<__nv_bfloat16, 64>, grid, 256, 0, st, false, a, kk, vv)
                     : launch(read_kernel<__nv_bfloat16, 128>, grid, 256, 0, st, false, a, kk, vv);
  }
  auto *kk = (float*)k, *vv = (float*)v;
  return g.d == 64 ? launch(read_kernel<float, 64>, grid, 256, 0, st, false, a, kk, vv)
                   : launch(read_kernel<float, 128>, grid, 256, 0, st, false, a, kk, vv);
}

namespace {
template <int D, int NT>
cudaError_t run_evict(const EvictArgs& a, size_t segs, cudaStream_t st) {
  static std::atomic<bool> once[64];
  const size_t words = (size_t)(a.max_rows + 31) / 32;
  const size_t smem = (2 * words + 1) * 4 + (a.max_rows <= kKeysInSmem ? (size_t)a.max_rows * 4 : 0);
  if (cudaError_t e = allow_smem((const void*)select_kernel<D, NT>, once, kSelectSmem)) return e;
  if (cudaError_t e = launch(select_kernel<D, NT>, dim3((unsigned)segs), NT, smem, st, false, a)) return e;
  return launch(move_kernel<D>, dim3((unsigned)((std::min(a.keep, a.max_rows) + kMove - 1) / kMove * segs)), 256, 0, st, true, a);
}
}  // namespace

cudaError_t kv4_evict(const Kv4Geom& g, int layer0, int n_layers, int n_seq, int max_rows, const int32_t* rows,
                      const int32_t* tables, const int32_t* next_pos, int keep, int recent, const int32_t* out_tables,
                      int out_pages, int32_t* rows_out, int32_t* status, void* ws, int num_sms, cudaStream_t st) {
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
  // Threads of a selection: few where rows are few (barriers cost less) or segments many (several CTAs share an SM, and
  // the long ones of a ragged batch still have warps enough).  Measured on ragged batches, both kernels (us, 256 / 512 /
  // 1,024 threads):
  //   rows 600:   128 segments 11 / 11 / 12,  512 segments 16 / 20 / 30,  2048 segments 43 / 51 / 95
  //   rows 2000:  128 segments 15 / 13 / 14,  512 segments 23 / 25 / 36,  2048 segments 64 / 72 / 120
  //   rows 8192:  128 segments 37 / 27 / 22,  512 segments 54 / 53 / 63,  2048 segments 183 / 180 / 248
  //   rows 16000: 128 segments 64 / 44 / 33,  512 segments 111 / 90 / 101
  const bool few = max_rows <= 1024, many = segs > (size_t)num_sms || max_rows <= 2048;
  if (g.d == 64) return few ? run_evict<64, 256>(a, segs, st) : many ? run_evict<64, 512>(a, segs, st) : run_evict<64, 1024>(a, segs, st);
  return few ? run_evict<128, 256>(a, segs, st) : many ? run_evict<128, 512>(a, segs, st) : run_evict<128, 1024>(a, segs, st);
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
