// mbk_kv4.cu -- a KV cache held in 4 bits: append, read, attention and eviction.
//
// A row of d elements (d 64 or 128) is held as groups of 64: codes 0 .. 15 in 4 bits and an fp16 pair
// (scale, lo); element = lo + scale * code.  Rows lie in blocks of 32 of one (layer, KV head), a block
// being contiguous: K codes [32][d / 2], K pairs [32][d / 64], V codes, V pairs and, in a tracked
// pool, positions int32 [32] and accumulated attention weights fp32 [32].
//
// Attention (attn_kernel).  A warp takes up to 8 (16) query rows -- (token, query head) pairs that
// read one KV head -- through a run of blocks.  With codes c and pairs (s, z) of row r
//     q . k_r = s_r (q . c_r) + z_r sum(q)        out = sum_r p_r s_r c_r + sum_r p_r z_r
// so the tensor cores multiply by the codes themselves and the pairs stay outside.  A code needs no
// conversion: its 4 bits in the low end of an fp16 are the subnormal code * 2^-24, exact as an operand
// of mma.sync; four bits higher it is 16 * code * 2^-24, and the 16 goes into q (QK) or the output's
// column (PV).  Eight codes of a 32-bit word become four operand registers with one shift and four
// ANDs (V, whose pairs run along rows: two more byte permutes per two words).  The tensor cores align a
// subnormal's products by its exponent field (2^-14), so a code in the low end gives up 6 bits or more of
// the sum's 24 (measured: 5e-5 off where 1e-6 was due); bf16 results do not notice, and for fp32 all codes
// are brought to the top of the subnormals, by three more shifts.
//   The operands stand as S^T = K Q^T and O^T = V^T P^T: 16 cache rows (16 dims) are the rows of the tile
// and the queries its 8 columns, so a KV head's few queries waste little.  The columns of S^T are
// those of O^T, so running maxima, sums and rescaling stay in a lane's own columns; between the two
// products P goes through one 8 x 8 transposition (movmatrix) per 8 rows.
//   fp32 queries keep fp32 accuracy: q is scaled to the top of fp16's range and split into
// hi + lo fp16 (22 bits), the softmax weights likewise; up to 4 queries hold hi in columns 0 .. 3 and lo
// in 4 .. 7, so that one mma does both, more take a second tile.  bf16 queries need one fp16 each.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "mbk_kv4.h"

namespace mbk {
namespace {

constexpr int kRows = kKv4Rows;
constexpr float kLog2e = 1.4426950408889634f;

// MODE: what a tile's columns hold.
enum Mode {
  BF16_8 = 0,   // 8 bf16 queries
  BF16_16 = 1,  // 16 bf16 queries, two tiles
  FP32_4 = 2,   // 4 fp32 queries: hi | lo
  FP32_8 = 3,   // 8 fp32 queries, a tile of hi and one of lo
};
// FEAT: 0: one token per sequence, nothing but the scale; 1: with cap or bias; 2: anything.  Only the last
// has rows that some columns of a tile see and others do not, whose NaNs must be kept from the others.

// Warps of an attention CTA (one CTA per SM) and blocks in flight per warp, within 227 KB of shared
// memory and 65,536 registers.
constexpr int kMaxWarps = 16;
template <int D, int MODE>
struct Shape {
  static constexpr int kGroups = D / 64;
  static constexpr int NT = MODE == BF16_16 || MODE == FP32_8 ? 2 : 1;  // tiles of 8 columns
  static constexpr int NS = MODE == BF16_16 ? 2 : 1;                    // column sets with a softmax of their own
  static constexpr int TILE = MODE == BF16_16 ? 16 : MODE == FP32_4 ? 4 : 8;
  static constexpr bool kPrecise = MODE >= FP32_4;
  static constexpr int kWarps = D == 64 ? 16 : NT == 2 ? 8 : 12;
  static constexpr int kStages = D == 64 && MODE != BF16_16 ? 4 : 3;
};

__device__ __forceinline__ void flag(int32_t* status, int bit) {
  if (status != nullptr) atomicOr(status, bit);
}

// ------------------------------------------------------------------ a sequence of a batch, bounds checked
struct SeqView {
  int r, c, tok0;  // rows of the cache, new tokens, first token
};
__device__ __forceinline__ SeqView seq_view(const Kv4Geom& g, const Kv4Batch& b, int s, bool report) {
  SeqView v;
  v.r = b.rows[s];
  v.tok0 = b.offsets[s];
  const int end = b.offsets[s + 1];
  bool bad = v.r < 0 || v.r > b.max_rows || v.tok0 < 0 || end < v.tok0 || end > b.n_tokens;
  if (bad) {
    v.r = min(max(v.r, 0), b.max_rows);
    v.tok0 = 0;
    v.c = 0;
  } else {
    v.c = end - v.tok0;
    if (v.c > b.max_count) {
      v.c = 0;
      bad = true;
    }
  }
  if (bad && report) flag(b.status, MBK_KV4_BAD_BATCH);
  return v;
}

// Start of the block that holds row `row` of the sequence with page table `table`, or null (and a
// status bit) when the table names a page outside the pool.
__device__ __forceinline__ uint8_t* block_of(const Kv4Geom& g, const int32_t* table, int layer, int h, int row, int32_t* status) {
  const int page = table[row >> g.page_shift];
  if ((unsigned)page >= (unsigned)g.num_pages) {
    flag(status, MBK_KV4_BAD_PAGE);
    return nullptr;
  }
  const int blk = (row & ((1 << g.page_shift) - 1)) / kRows;
  return g.pool + (size_t)page * g.page_stride + (size_t)(layer * g.nkv + h) * g.head_stride + (size_t)blk * g.block_bytes;
}

// Byte offsets of a block's fields.
__host__ __device__ constexpr int code_bytes(int d) { return kRows * d / 2; }
__host__ __device__ constexpr int pair_bytes(int d) { return kRows * d / 64 * 4; }
__host__ __device__ constexpr int half_bytes(int d) { return code_bytes(d) + pair_bytes(d); }  // K or V
__host__ __device__ constexpr int pos_at(int d) { return 2 * half_bytes(d); }
__host__ __device__ constexpr int weight_at(int d) { return 2 * half_bytes(d) + 4 * kRows; }

// ------------------------------------------------------------------ append and read
// Eight lanes hold a group of 64, 8 elements each; a block of threads takes `per` tokens of one
// sequence (grid.y).  Bound by the bytes: 8 n d elements read, 0.56 bytes written for each.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
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

// ------------------------------------------------------------------ attention: the work and its split
// A segment is one (sequence, KV head, tile of query rows); its units are the blocks of 32 cache rows
// that it reads.  All segments' units, in order, are cut into equal runs, one per CTA and within it one
// per warp, whatever the sequences' lengths: a long context is spread over all SMs and a batch of
// short ones leaves none idle.  A segment inside one warp's run is written by the warp, one inside a
// CTA's run is joined in shared memory, the rest is joined by combine_kernel.
struct SeqInfo {
  int cum, r, c, tok0;  // units before the sequence; rows, new tokens, first token
};

struct AttnArgs {
  Kv4Geom g;
  Kv4Batch b;
  Kv4Attn a;
  int layer, grp, grid_max, warps;
  float cap2;    // 2 log2(e) / cap
  float* part;   // [grid][2][tile rows][d + 2] partial (o, m, l) of segments that several CTAs share
  float* lse;    // [n_tokens][nq] log2 of the softmax denominators (accumulate), or null
};

template <int TILE>
struct Split {
  int n_seq, nkv, grp, window, track, total, grid;
  const SeqInfo* seq;

  __device__ int first_block(const SeqInfo& q) const {
    return window > 0 && !track ? max(0, q.r - q.c - window + 1) / kRows : 0;
  }
  __device__ int blocks(const SeqInfo& q) const { return max(1, (q.r + kRows - 1) / kRows - first_block(q)); }
  __device__ int tiles(const SeqInfo& q) const { return (q.c * grp + TILE - 1) / TILE; }
  __device__ int units(const SeqInfo& q) const { return q.c == 0 ? 0 : tiles(q) * nkv * blocks(q); }
  // the run of CTA i
  __device__ int begin(int i) const { return (int)((long long)total * i / grid); }
  __device__ int cta_of(int u) const {
    int i = (int)((long long)u * grid / total);
    while (i + 1 < grid && begin(i + 1) <= u) ++i;
    while (i > 0 && begin(i) > u) --i;
    return i;
  }
};

// Fills info[0 .. n_seq - 1] (cum of entry n_seq - 1 included) and returns the split; all threads call.
template <int TILE>
__device__ Split<TILE> make_split(const AttnArgs& a, SeqInfo* info, int* warp_sums, bool report) {
  Split<TILE> sp;
  sp.n_seq = a.b.n_seq;
  sp.nkv = a.g.nkv;
  sp.grp = a.grp;
  sp.window = a.a.window;
  sp.track = a.g.track;
  sp.seq = info;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int carry = 0;
  for (int s0 = 0; s0 < a.b.n_seq; s0 += blockDim.x) {
    const int s = s0 + threadIdx.x;
    SeqInfo q{0, 0, 0, 0};
    int n = 0;
    if (s < a.b.n_seq) {
      const SeqView v = seq_view(a.g, a.b, s, report);
      q.r = v.r;
      q.c = v.c;
      q.tok0 = v.tok0;
      n = sp.units(q);
    }
    int x = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, m);
      if (lane >= m) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = carry, all = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) before += warp_sums[w];
      all += warp_sums[w];
    }
    q.cum = before + x - n;
    if (s < a.b.n_seq) info[s] = q;
    carry += all;
    __syncthreads();
  }
  sp.total = carry;
  // one block for each warp of a CTA before a second CTA is used
  sp.grid = max(1, min(a.grid_max, (carry + a.warps - 1) / a.warps));
  return sp;
}

struct Seg {
  int s, h, tile, first, n, u0;  // sequence, KV head, tile; first block, blocks, first unit
};
template <int TILE>
__device__ Seg locate(const Split<TILE>& sp, int u) {
  int lo = 0, hi = sp.n_seq - 1;
  while (lo < hi) {  // last sequence with cum <= u (those without units share the next one's cum)
    const int mid = (lo + hi + 1) >> 1;
    if (sp.seq[mid].cum <= u) lo = mid; else hi = mid - 1;
  }
  const SeqInfo q = sp.seq[lo];
  Seg g;
  g.s = lo;
  g.first = sp.first_block(q);
  g.n = sp.blocks(q);
  const int rem = u - q.cum, i = rem / g.n, nt = sp.tiles(q);
  g.h = i / nt;
  g.tile = i - g.h * nt;
  g.u0 = q.cum + i * g.n;
  return g;
}

// ------------------------------------------------------------------ attention: one block of 32 rows
__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// d = a b + c on a 16 x 8 x 16 tile of fp16 with fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// The transpose of the 8 x 8 matrix of 16-bit values of which this lane holds row gid, columns 2 tig, 2 tig + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// (a, b) += (c, d) in one instruction.
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b) : "f"(c), "f"(d));
}
// The codes of a word as four operand registers (codes i and i + 4 in register i), in units of
// 2^-24 (16 times that in registers 1 and 3), with PRECISE of 2^-18.
template <bool PRECISE>
__device__ __forceinline__ void codes(uint32_t x, uint32_t (&r)[4]) {
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kTop = 0x03c003c0u;
  if (PRECISE) {
    r[0] = (x << 6) & kTop;
    r[1] = (x << 2) & kTop;
    r[2] = (x >> 2) & kTop;
    r[3] = (x >> 6) & kTop;
  } else {
    const uint32_t x8 = x >> 8;
    r[0] = x & kLow;
    r[1] = x & kHigh;
    r[2] = x8 & kLow;
    r[3] = x8 & kHigh;
  }
}
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// A stage of the ring in shared memory: per group of 64 dims, 32 rows of 32 bytes.  Lane (gid, tig) of
// the mma fragments reads 8 bytes of K rows 4 gid + i (so its rows' pairs are contiguous) and 4 bytes of
// V rows 8 tig + i; row r goes to byte (r % 8) * 128 + ((r / 8) ^ 2 (r / 4 % 2)) * 32, which makes both
// free of bank conflicts.
__device__ __forceinline__ int place(int r) { return (r & 7) * 128 + (((r >> 3) ^ ((r & 4) >> 1)) << 5); }

template <int D>
struct Stage {
  static constexpr int kGroups = D / 64;
  static constexpr int kCodes = kGroups * 1024, kPairs = kGroups * 128;
  static constexpr int kV = kCodes + kPairs;        // K codes, K pairs, V codes, V pairs, positions
  static constexpr int kPos = 2 * kV;
  static constexpr int kBytes = 2 * kV + 128;
};

template <int D>
__device__ __forceinline__ void fetch(uint32_t st, const uint8_t* blk, bool pos, int lane) {
  using S = Stage<D>;
  constexpr int kGroups = S::kGroups;
#pragma unroll
  for (int sel = 0; sel < 2; ++sel) {
    const uint8_t* src = blk + sel * half_bytes(D);
#pragma unroll
    for (int i = 0; i < 2 * kGroups; ++i) {
      const int c = i * 32 + lane, r = c / (2 * kGroups), in = c % (2 * kGroups);
      cp16(st + sel * S::kV + (in >> 1) * 1024 + place(r) + (in & 1) * 16, src + c * 16);
    }
  }
  // the pairs: kGroups * 8 chunks each of K and V, then the positions
  if (lane < 16 * kGroups) {
    const int sel = lane / (8 * kGroups), c = lane % (8 * kGroups);
    cp16(st + sel * S::kV + S::kCodes + c * 16, blk + sel * half_bytes(D) + code_bytes(D) + c * 16);
  }
  if (pos && lane < 8) cp16(st + S::kPos + lane * 16, blk + pos_at(D) + lane * 16);
}

// The queries of a tile as B fragments, and per lane what belongs to its columns 2 tig and 2 tig + 1.
template <int D, int MODE>
struct QTile {
  using P = Shape<D, MODE>;
  uint32_t f[P::kGroups][4][P::NT][2];
  float mul[P::NS][2], add[P::kGroups][P::NS][2];  // score = scale_r * acc * mul + z_r * add, natural logarithm's units
  float mid[P::kGroups][2];                        // fp32: -7.5 sum(q) in acc's units; codes count from their middle
  int limit[P::NS][2], qpos[P::NS][2];             // last visible row (-1: none), position
  float slope[P::NS][2];
};

// Query column of a lane's C column j of softmax set ns.
template <int MODE>
__device__ __forceinline__ int column(int tig, int ns, int j) {
  return MODE == FP32_4 ? (2 * tig + j) & 3 : 8 * ns + 2 * tig + j;
}

template <int D, int MODE, int FEAT>
__device__ __forceinline__ void load_q(QTile<D, MODE>& t, const AttnArgs& a, const SeqInfo& sq, int s, int h, int tile, int lane) {
  using P = Shape<D, MODE>;
  constexpr int kGroups = P::kGroups, NS = P::NS;
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int ns = 0; ns < NS; ++ns) {
    // this lane: column gid, dims 16 tig .. + 15 of each group
    const int col = MODE == FP32_4 ? gid & 3 : 8 * ns + gid;
    const int row = tile * P::TILE + col, tok = row / a.grp, head = h * a.grp + row - tok * a.grp;
    const bool on = tok < sq.c;
    float x[kGroups][16], sum[kGroups];
    float mx = 0.f;
    const size_t at = (size_t)(sq.tok0 + tok) * a.a.ldq + (size_t)head * D + 16 * tig;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      sum[g] = 0.f;
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (on) {
          if (P::kPrecise) load8<float>(reinterpret_cast<const float*>(a.a.q) + at + 64 * g + 8 * v, y);
          else load8<__nv_bfloat16>(reinterpret_cast<const __nv_bfloat16*>(a.a.q) + at + 64 * g + 8 * v, y);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[g][8 * v + i] = y[i];
          mx = fmaxf(mx, fabsf(y[i]));
          sum[g] += y[i];
        }
      }
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // the row's largest element to [2^13, 2^14): fp16 then keeps 22 bits of all that matters in hi + lo
    int ex = (__float_as_int(mx) >> 23) & 255;
    ex = ex == 255 ? 140 : max(ex, 20);
    const float up = pow2i(140 - ex);
    const float up0 = P::kPrecise ? up / 64.f : up, up1 = P::kPrecise ? up0 : up / 16.f;  // the codes' units
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        // k step ks = 2 w + y: word w's code pairs (2 y, 2 y + 4) and (2 y + 1, 2 y + 5)
        const int w = ks >> 1, y = ks & 1;
        const float e0 = x[g][8 * w + 2 * y] * up0, e1 = x[g][8 * w + 2 * y + 4] * up0;
        const float e2 = x[g][8 * w + 2 * y + 1] * up1, e3 = x[g][8 * w + 2 * y + 5] * up1;
        const uint32_t h0 = pack_half(e0, e1), h1 = pack_half(e2, e3);
        if (P::kPrecise) {
          const float2 u0 = unpack_half(h0), u1 = unpack_half(h1);
          const uint32_t l0 = pack_half(e0 - u0.x, e1 - u0.y), l1 = pack_half(e2 - u1.x, e3 - u1.y);
          if (MODE == FP32_4) {
            t.f[g][ks][0][0] = gid < 4 ? h0 : l0;
            t.f[g][ks][0][1] = gid < 4 ? h1 : l1;
          } else {
            t.f[g][ks][0][0] = h0;
            t.f[g][ks][0][1] = h1;
            t.f[g][ks][P::NT - 1][0] = l0;
            t.f[g][ks][P::NT - 1][1] = l1;
          }
        } else {
          t.f[g][ks][ns][0] = h0;
          t.f[g][ks][ns][1] = h1;
        }
      }
    const float down = pow2i(ex - 140) * 16777216.f;  // 2^24: the codes' subnormal unit
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int from = 4 * (2 * tig + j);  // a lane of that column
      t.mul[ns][j] = __shfl_sync(0xffffffffu, down, from) * a.a.scale;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float sg = __shfl_sync(0xffffffffu, sum[g], from);
        t.add[g][ns][j] = sg * a.a.scale;
        if (P::kPrecise) {
          const float m = sg * (-7.5f / 16777216.f) * __shfl_sync(0xffffffffu, up, from);
          t.mid[g][j] = MODE == FP32_4 && tig >= 2 ? 0.f : m;  // the lo columns start at zero
        }
      }
      const int crow = tile * P::TILE + column<MODE>(tig, ns, j), ctok = crow / a.grp;
      const bool con = ctok < sq.c;
      t.limit[ns][j] = con ? sq.r - sq.c + ctok : -1;
      if (FEAT > 0) {
        t.qpos[ns][j] = con ? (a.b.positions != nullptr ? a.b.positions[s] : sq.r - sq.c) + ctok : 0;
        t.slope[ns][j] = con && a.a.slopes != nullptr ? a.a.slopes[h * a.grp + crow - ctok * a.grp] : 0.f;
      }
    }
  }
}

// Scores of the tile against a staged block, in units of the base-2 logarithm: sc[ns][i][j] is cache row
// 32 blk + 4 gid + i against the lane's column j of set ns; -inf where the row is not visible.
// full: every row of the block is visible to every query of the tile (a window aside).
template <int D, int MODE, int FEAT>
__device__ __forceinline__ void scores(const QTile<D, MODE>& t, const AttnArgs& a, const unsigned char* st, int blk, bool full, int lane,
                                       float (&sc)[Shape<D, MODE>::NS][4][2]) {
  using S = Stage<D>;
  using P = Shape<D, MODE>;
  constexpr int kGroups = P::kGroups, NS = P::NS, NT = P::NT;
  const int gid = lane >> 2, tig = lane & 3;
  uint32_t pr[kGroups * 4];
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    *reinterpret_cast<uint4*>(pr + 4 * i) = *reinterpret_cast<const uint4*>(st + S::kCodes + gid * (16 * kGroups) + 16 * i);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {  // tile rows gid: cache row 4 gid + 2 mt; gid + 8: the next one
      const uint2 w0 = *reinterpret_cast<const uint2*>(st + g * 1024 + place(4 * gid + 2 * mt) + 8 * tig);
      const uint2 w1 = *reinterpret_cast<const uint2*>(st + g * 1024 + place(4 * gid + 2 * mt + 1) + 8 * tig);
      float c[NT][4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t x[4], y[4];
        codes<P::kPrecise>(k ? w0.y : w0.x, x);
        codes<P::kPrecise>(k ? w1.y : w1.x, y);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t af[4] = {x[2 * z], y[2 * z], x[2 * z + 1], y[2 * z + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint32_t(&b)[2] = t.f[g][2 * k + z][nt];
            if (k + z > 0) mma(c[nt], af, b[0], b[1], c[nt][0], c[nt][1], c[nt][2], c[nt][3]);
            else if (P::kPrecise && nt == 0) mma(c[nt], af, b[0], b[1], t.mid[g][0], t.mid[g][1], t.mid[g][0], t.mid[g][1]);
            else mma(c[nt], af, b[0], b[1], 0.f, 0.f, 0.f, 0.f);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 p = unpack_half(pr[(2 * mt + i) * kGroups + g]);
        const float z = P::kPrecise ? fmaf(7.5f, p.x, p.y) : p.y;
#pragma unroll
        for (int ns = 0; ns < NS; ++ns)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float acc = c[ns][2 * i + j];
            if (MODE == FP32_8) acc += c[NT - 1][2 * i + j];
            if (MODE == FP32_4) acc += __shfl_xor_sync(0xffffffffu, acc, 2);
            const float x = fmaf(p.x, acc * t.mul[ns][j], z * t.add[g][ns][j]);
            if (g == 0) sc[ns][2 * mt + i][j] = x;
            else sc[ns][2 * mt + i][j] += x;
          }
      }
    }
  }
  const int r0 = blk * kRows + 4 * gid;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int kpos = FEAT > 0 && a.g.track ? *reinterpret_cast<const int*>(st + S::kPos + 4 * (4 * gid + i)) : r0 + i;
#pragma unroll
    for (int ns = 0; ns < NS; ++ns)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = sc[ns][i][j];
        bool see = full || r0 + i <= t.limit[ns][j];
        if (FEAT > 0) {
          if (a.a.cap > 0.f) {
            // cap tanh(x / cap) = cap (1 - 2 / (1 + exp(2 x / cap))): off by a few 2^-24 of cap
            const float e = ex2(fminf(x * a.cap2, 126.f));
            x = a.a.cap * (1.f - __fdividef(2.f, 1.f + e));
          }
          const int gap = kpos - t.qpos[ns][j];
          if (a.a.slopes != nullptr) x = fmaf(t.slope[ns][j], (float)gap, x);
          if (FEAT == 2 && a.a.window > 0) see = see && gap > -a.a.window;
        }
        sc[ns][i][j] = see ? x * kLog2e : -INFINITY;
      }
  }
}

// Running softmax and output of a tile.  The reference value m of a column is a maximum of its scores that
// is only renewed when a score exceeds it by kSlack (a factor of 256 in the weight): until then no lane needs
// to know another's maximum, and nothing is rescaled.
constexpr float kSlack = 8.f;
constexpr int kUnit = 6;  // weights are held as p * scale_r * 2^(kUnit - e): below 2^15
template <int D, int MODE>
struct Acc {
  using P = Shape<D, MODE>;
  float o[P::kGroups][4][P::NT][4];  // dims 8 gid + 2 mt + {0, 1}, columns 2 tig + {0, 1}; units: 2^(kUnit - e) times those of codes()
  float m[P::NS][2], l[P::NS][2], z[P::kGroups][P::NS][2];  // l and z: this lane's rows only
  int e;                             // exponent of the largest scale of V seen so far
  __device__ void clear() {
#pragma unroll
    for (int g = 0; g < P::kGroups; ++g)
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < P::NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[g][mt][nt][k] = 0.f;
#pragma unroll
    for (int ns = 0; ns < P::NS; ++ns)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[ns][j] = -INFINITY;
        l[ns][j] = 0.f;
#pragma unroll
        for (int g = 0; g < P::kGroups; ++g) z[g][ns][j] = 0.f;
      }
    e = -24;
  }
};

template <int D, int MODE, int FEAT>
__device__ __forceinline__ void accumulate(Acc<D, MODE>& A, const unsigned char* st, int blk, int rows, int lane,
                                           float (&sc)[Shape<D, MODE>::NS][4][2]) {
  using S = Stage<D>;
  using P = Shape<D, MODE>;
  constexpr int kGroups = P::kGroups, NS = P::NS, NT = P::NT;
  const int gid = lane >> 2, tig = lane & 3;
  uint32_t pr[kGroups * 4];
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    *reinterpret_cast<uint4*>(pr + 4 * i) = *reinterpret_cast<const uint4*>(st + S::kV + S::kCodes + gid * (16 * kGroups) + 16 * i);
  if ((blk + 1) * kRows > rows) {  // rows behind the cache's end hold anything, NaN among it
    const int r0 = blk * kRows + 4 * gid;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r0 + i >= rows) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) pr[i * kGroups + g] = 0u;
      }
  }
  __half2 mx = *reinterpret_cast<const __half2*>(&pr[0]);
#pragma unroll
  for (int i = 1; i < 4 * kGroups; ++i) mx = __hmax2(mx, *reinterpret_cast<const __half2*>(&pr[i]));
  const int eb = min((int)((*reinterpret_cast<const uint32_t*>(&mx) >> 10) & 31u) - 15, 15);  // of the largest scale (low halves)
  bool over = eb > A.e;
#pragma unroll
  for (int ns = 0; ns < NS; ++ns)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      over = over || fmaxf(fmaxf(sc[ns][0][j], sc[ns][1][j]), fmaxf(sc[ns][2][j], sc[ns][3][j])) > A.m[ns][j] + kSlack;
  if (__any_sync(0xffffffffu, over)) {
    const int e = max(A.e, (int)__reduce_max_sync(0xffffffffu, (unsigned)(eb + 32)) - 32);
    const float unit = pow2i(A.e - e);
    A.e = e;
    float al[NS][2];
#pragma unroll
    for (int ns = 0; ns < NS; ++ns)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float bm = fmaxf(fmaxf(sc[ns][0][j], sc[ns][1][j]), fmaxf(sc[ns][2][j], sc[ns][3][j]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, x));
        const float nm = fmaxf(A.m[ns][j], bm);
        al[ns][j] = nm == -INFINITY ? 1.f : ex2(A.m[ns][j] - nm);
        A.m[ns][j] = nm;
        A.l[ns][j] *= al[ns][j];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) A.z[g][ns][j] *= al[ns][j];
        al[ns][j] *= unit;
      }
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) A.o[g][mt][nt][k] *= al[NS == 2 ? nt : 0][k & 1];
  }
#pragma unroll
  for (int ns = 0; ns < NS; ++ns)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float base = A.m[ns][j] == -INFINITY ? 0.f : A.m[ns][j];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[ns][i][j] = ex2(sc[ns][i][j] - base);
        A.l[ns][j] += sc[ns][i][j];
      }
    }
  const float f = pow2i(kUnit - A.e);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    uint32_t bf[NT][4];  // P^T as B fragments: register i holds rows 8 tig + i and 8 tig + 4 + i of column gid
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack_half(pr[i * kGroups + g]);
      const float z = P::kPrecise ? fmaf(p.x, 7.5f, p.y) : p.y, sf = p.x * f;
#pragma unroll
      for (int ns = 0; ns < NS; ++ns) {
        float x[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float w = sc[ns][i][j];
          if (FEAT == 2) {  // a weight of zero (a masked row) takes nothing of its row, NaN included
            x[j] = w > 0.f ? w * sf : w;
            A.z[g][ns][j] += w > 0.f ? w * z : w;
          } else {
            x[j] = w * sf;
            A.z[g][ns][j] = fmaf(w, z, A.z[g][ns][j]);
          }
        }
        const uint32_t hi = pack_half(x[0], x[1]);
        if (P::kPrecise) {
          const float2 u = unpack_half(hi);
          const uint32_t lo = pack_half(x[0] - u.x, x[1] - u.y);
          if (MODE == FP32_4) {
            bf[0][i] = transpose8(tig < 2 ? hi : lo);
          } else {
            bf[0][i] = transpose8(hi);
            bf[NT - 1][i] = transpose8(lo);
          }
        } else {
          bf[ns][i] = transpose8(hi);
        }
      }
    }
    // The block's share is summed from zero and added in fp32: the tensor cores' own sums are truncated, and
    // over thousands of rows that bias showed (3e-4).  For fp32 they also start at -7.5 sum(p), so that
    // codes count from their middle: sum p (code - 7.5) is of the output's size, sum p code many times that.
    float mid[NT][4];
    if (P::kPrecise) {
      constexpr uint32_t kMinus = 0x81e081e0u;  // -480 * 2^-24: -7.5 in units of 2^-18
      constexpr uint32_t am[4] = {kMinus, kMinus, kMinus, kMinus};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma(mid[nt], am, bf[nt][0], bf[nt][1], 0.f, 0.f, 0.f, 0.f);
        mma(mid[nt], am, bf[nt][2], bf[nt][3], mid[nt][0], mid[nt][1], mid[nt][2], mid[nt][3]);
      }
    }
    const unsigned char* vb = st + S::kV + g * 1024 + 4 * gid;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(vb + place(8 * tig + i));
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // codes 4 half .. + 3 of the word: dims 8 gid + 4 half ..
      const uint32_t sel = half ? 0x7632u : 0x5410u;
      uint32_t x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) codes<P::kPrecise>(__byte_perm(w[i], w[i + 4], sel), x[i]);
#pragma unroll
      for (int m2 = 0; m2 < 2; ++m2)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t a0[4] = {x[0][2 * m2], x[0][2 * m2 + 1], x[1][2 * m2], x[1][2 * m2 + 1]};
          const uint32_t a1[4] = {x[2][2 * m2], x[2][2 * m2 + 1], x[3][2 * m2], x[3][2 * m2 + 1]};
          float c[4];
          if (P::kPrecise) mma(c, a0, bf[nt][0], bf[nt][1], mid[nt][0], mid[nt][1], mid[nt][2], mid[nt][3]);
          else mma(c, a0, bf[nt][0], bf[nt][1], 0.f, 0.f, 0.f, 0.f);
          mma(c, a1, bf[nt][2], bf[nt][3], c[0], c[1], c[2], c[3]);
          float(&o)[4] = A.o[g][2 * half + m2][nt];
          add2(o[0], o[1], c[0], c[1]);
          add2(o[2], o[3], c[2], c[3]);
        }
    }
  }
}

__device__ __forceinline__ void store_out(const Kv4Attn& a, size_t at, const float (&x)[8]) {
  if (a.bf16) store8(reinterpret_cast<__nv_bfloat16*>(a.out) + at, x);
  else store8(reinterpret_cast<float*>(a.out) + at, x);
}
__device__ __forceinline__ float all_rows(float x) {  // sum over the lanes of a column
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// The end of a tile's run: the sums over the columns' lanes; then either the output itself or the
// partial (o [d], m, l) of each column at `dep` (d + 2 floats apart).
template <int D, int MODE>
__device__ __forceinline__ void finish(Acc<D, MODE>& A, const AttnArgs& a, const SeqInfo& sq, int h, int tile, int lane, float* dep) {
  using P = Shape<D, MODE>;
  constexpr int NS = P::NS;
  const int gid = lane >> 2, tig = lane & 3;
  const float unit = pow2i(A.e - kUnit + 24);
  const float u0 = P::kPrecise ? unit / 64.f : unit, u1 = P::kPrecise ? u0 : unit / 16.f;
#pragma unroll
  for (int ns = 0; ns < NS; ++ns)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float l = all_rows(A.l[ns][j]);
      const int col = column<MODE>(tig, ns, j), row = tile * P::TILE + col, tok = row / a.grp, head = h * a.grp + row - tok * a.grp;
      const bool on = tok < sq.c && !(MODE == FP32_4 && tig >= 2);
      const float inv = dep != nullptr ? 1.f : (l > 0.f || l != l ? 1.f / l : 0.f);
#pragma unroll
      for (int g = 0; g < P::kGroups; ++g) {
        const float z = all_rows(A.z[g][ns][j]);
        float x[8];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float o = A.o[g][mt][NS == 2 ? ns : 0][2 * y + j];
            if (MODE == FP32_8) o += A.o[g][mt][P::NT - 1][2 * y + j];
            if (MODE == FP32_4) o += __shfl_xor_sync(0xffffffffu, o, 2);
            x[2 * mt + y] = fmaf(o, y ? u1 : u0, z) * inv;
          }
        if (!on) continue;
        if (dep != nullptr) {
          float* d = dep + col * (D + 2) + 64 * g + 8 * gid;
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = x[i];
        } else {
          store_out(a.a, (size_t)(sq.tok0 + tok) * a.a.ldo + (size_t)head * D + 64 * g + 8 * gid, x);
        }
      }
      if (on && gid == 0) {
        if (dep != nullptr) {
          dep[col * (D + 2) + D] = A.m[ns][j];
          dep[col * (D + 2) + D + 1] = l;
        } else if (a.lse != nullptr) {
          a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] = l > 0.f ? A.m[ns][j] + log2f(l) : INFINITY;
        }
      }
    }
}

template <int D, int MODE, int FEAT>
__global__ void __launch_bounds__(Shape<D, MODE>::kWarps * 32) attn_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int TILE = Shape<D, MODE>::TILE, kWarps = Shape<D, MODE>::kWarps, kStages = Shape<D, MODE>::kStages;
  static_assert(kStages * Stage<D>::kBytes >= TILE * (D + 2) * 4, "a warp's last partial lies in its ring");
  using S = Stage<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int warp_sums[kWarps];
  __shared__ int dep_seg[kWarps][2];  // first unit of the segment of a warp's partial, or -1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SeqInfo* info = reinterpret_cast<SeqInfo*>(smem);
  unsigned char* ring = smem + ((size_t)a.b.n_seq * sizeof(SeqInfo) + 127) / 128 * 128;
  // a warp's first partial (its run goes on) beside the rings, its last one in its own ring
  float* deps = reinterpret_cast<float*>(ring + (size_t)kWarps * kStages * S::kBytes);
  const int dep_floats = min(TILE, a.b.max_count * a.grp) * (D + 2);
  auto dep_at = [&](int k) {  // k = 2 warp + slot
    return (k & 1) ? reinterpret_cast<float*>(ring + (size_t)(k >> 1) * kStages * S::kBytes) : deps + (size_t)(k >> 1) * dep_floats;
  };
  const Split<TILE> sp = make_split<TILE>(a, info, warp_sums, blockIdx.x == 0);
  if (lane < 2) dep_seg[warp][lane] = -1;
  __syncthreads();
  if ((int)blockIdx.x >= sp.grid || sp.total == 0) return;
  const int c0 = sp.begin(blockIdx.x), c1 = sp.begin(blockIdx.x + 1), cn = c1 - c0;
  const int u0 = c0 + (int)((long long)cn * warp / kWarps), u1 = c0 + (int)((long long)cn * (warp + 1) / kWarps);
  unsigned char* mine = ring + (size_t)warp * kStages * S::kBytes;
  const uint32_t mine_s = smem_of(mine);

  if (u0 < u1) {
    const bool need_pos = FEAT > 0 && a.g.track;
    Seg ps = locate(sp, u0);  // the copies' segment
    Seg cs = ps;              // the arithmetic's
    SeqInfo psq = info[ps.s], csq = psq;
    unsigned have = 0;        // bit i: stage i holds a block to be used
    auto last_row = [&](const Seg& g, const SeqInfo& q) {  // last row that any query of the tile sees
      const int tok = min(q.c - 1, (g.tile * TILE + TILE - 1) / a.grp);
      return q.r - q.c + tok;
    };
    int plast = last_row(ps, psq);
    auto issue = [&](int u) {
      if (u < u1) {
        if (u >= ps.u0 + ps.n) {
          ps = locate(sp, u);
          psq = info[ps.s];
          plast = last_row(ps, psq);
        }
        const int blk = ps.first + u - ps.u0, stg = (u - u0) % kStages;
        have &= ~(1u << stg);
        if (blk * kRows <= plast) {
          const uint8_t* p = block_of(a.g, a.b.tables + (size_t)ps.s * a.g.max_pages, a.layer, ps.h, blk * kRows,
                                      lane == 0 ? a.b.status : nullptr);
          if (p != nullptr) {
            have |= 1u << stg;
            fetch<D>(mine_s + stg * S::kBytes, p, need_pos, lane);
          }
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(u0 + i);
    QTile<D, MODE> qt;
    Acc<D, MODE> acc;
    int u = u0;
    while (u < u1) {
      if (u != u0) {
        cs = locate(sp, u);
        csq = info[cs.s];
      }
      load_q<D, MODE, FEAT>(qt, a, csq, cs.s, cs.h, cs.tile, lane);
      acc.clear();
      const int first_limit = csq.r - csq.c + (cs.tile * TILE) / a.grp;
      const int end = min(u1, cs.u0 + cs.n);
      for (; u < end; ++u) {
        cp_wait<kStages - 2>();
        __syncwarp();
        const int stg = (u - u0) % kStages, blk = cs.first + u - cs.u0;
        const bool use = (have >> stg) & 1u;
        issue(u + kStages - 1);  // into the stage that the iteration before has read
        if (use) {
          const unsigned char* st = mine + stg * S::kBytes;
          float sc[Shape<D, MODE>::NS][4][2];
          scores<D, MODE, FEAT>(qt, a, st, blk, (blk + 1) * kRows - 1 <= first_limit, lane, sc);
          accumulate<D, MODE, FEAT>(acc, st, blk, csq.r, lane, sc);
        }
        __syncwarp();
      }
      const bool whole = cs.u0 >= u0 && cs.u0 + cs.n <= u1;
      if (whole) {
        finish<D, MODE>(acc, a, csq, cs.h, cs.tile, lane, nullptr);
      } else {
        const int slot = cs.u0 < u0 ? 0 : 1;  // it began in an earlier warp's run, or goes on in a later one's
        if (lane == 0) dep_seg[warp][slot] = cs.u0;
        finish<D, MODE>(acc, a, csq, cs.h, cs.tile, lane, dep_at(2 * warp + slot));
      }
    }
  }
  __syncthreads();
  // join the warps' partials, segment by segment (they lie in the order of the warps)
  for (int i = 0; i < 2 * kWarps;) {
    const int seg = dep_seg[i >> 1][i & 1];
    if (seg < 0) {
      ++i;
      continue;
    }
    int j = i + 1;
    while (j < 2 * kWarps && (dep_seg[j >> 1][j & 1] < 0 || dep_seg[j >> 1][j & 1] == seg)) ++j;
    const Seg g = locate(sp, seg);
    const SeqInfo sq = info[g.s];
    const bool inside = g.u0 >= c0 && g.u0 + g.n <= c1;
    const int nrow = min(TILE, sq.c * a.grp - g.tile * TILE);
    float* out = a.part + ((size_t)blockIdx.x * 2 + (g.u0 < c0 ? 0 : 1)) * TILE * (D + 2);
    for (int x = threadIdx.x; x < nrow * (D / 8); x += blockDim.x) {
      const int row = x / (D / 8), d0 = x % (D / 8) * 8;
      float m = -INFINITY;
      for (int k = i; k < j; ++k)
        if (dep_seg[k >> 1][k & 1] >= 0) m = fmaxf(m, dep_at(k)[row * (D + 2) + D]);
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k = i; k < j; ++k)
        if (dep_seg[k >> 1][k & 1] >= 0) {
          const float* p = dep_at(k) + row * (D + 2);
          const float w = ex2(p[D] - base);
          l = fmaf(p[D + 1], w, l);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(p[d0 + e], w, o[e]);
        }
      const int tr = g.tile * TILE + row, tok = tr / a.grp, head = g.h * a.grp + tr - tok * a.grp;
      if (inside) {
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= inv;
        store_out(a.a, (size_t)(sq.tok0 + tok) * a.a.ldo + (size_t)head * D + d0, o);
        if (a.lse != nullptr && d0 == 0) a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] = l > 0.f ? m + log2f(l) : INFINITY;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) out[row * (D + 2) + d0 + e] = o[e];
        if (d0 == 0) {
          out[row * (D + 2) + D] = m;
          out[row * (D + 2) + D + 1] = l;
        }
      }
    }
    i = j;
  }
}

// Joins the partials of segments that several CTAs share; grid: (KV heads x tiles at most, sequences).
template <int D, int TILE>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int warp_sums[kMaxWarps];
  SeqInfo* info = reinterpret_cast<SeqInfo*>(smem);
  const Split<TILE> sp = make_split<TILE>(a, info, warp_sums, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (sp.total == 0) return;
  const SeqInfo sq = info[blockIdx.y];
  const int nt = sp.tiles(sq), n = sp.blocks(sq);
  for (int i = blockIdx.x; i < nt * a.g.nkv; i += gridDim.x) {
    const int u0 = sq.cum + i * n, first = sp.cta_of(u0), last = sp.cta_of(u0 + n - 1);
    if (first == last) continue;
    const int h = i / nt, tile = i - h * nt;
    const int nrow = min(TILE, sq.c * a.grp - tile * TILE);
    for (int x = threadIdx.x; x < nrow * (D / 8); x += blockDim.x) {
      const int row = x / (D / 8), d0 = x % (D / 8) * 8;
      auto part = [&](int k) { return a.part + (((size_t)k * 2 + (k == first ? 1 : 0)) * TILE + row) * (D + 2); };
      float m = -INFINITY;
      for (int k = first; k <= last; ++k) m = fmaxf(m, part(k)[D]);
      const float base = m == -INFINITY ? 0.f : m;
      float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int k = first; k <= last; ++k) {
        const float* p = part(k);
        const float w = ex2(p[D] - base);
        l = fmaf(p[D + 1], w, l);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = fmaf(p[d0 + e], w, o[e]);
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= inv;
      const int tr = tile * TILE + row, tok = tr / a.grp, head = h * a.grp + tr - tok * a.grp;
      store_out(a.a, (size_t)(sq.tok0 + tok) * a.a.ldo + (size_t)head * D + d0, o);
      if (a.lse != nullptr && d0 == 0) a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] = l > 0.f ? m + log2f(l) : INFINITY;
    }
  }
}

// The weight that each cache row got: weight_r += sum over the sequence's queries and the group's heads
// of exp2(score - lse).  A warp owns a block's 32 rows and goes through all the query tiles, so the
// sums have one order and no atomics; the scores are computed again from K (half a row's bytes)
// rather than kept, which would cost 4 bytes written and read for each of the group's heads.
template <int D, int MODE, int FEAT>
__global__ void __launch_bounds__(256) weight_kernel(const __grid_constant__ AttnArgs a) {
  using P = Shape<D, MODE>;
  using S = Stage<D>;
  constexpr int TILE = P::TILE;
  extern __shared__ __align__(128) unsigned char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int s = blockIdx.z, h = blockIdx.y;
  const SeqView v = seq_view(a.g, a.b, s, false);
  if (v.c == 0) return;
  const SeqInfo sq{0, v.r, v.c, v.tok0};
  unsigned char* st = smem + warp * S::kBytes;
  const int nblk = (v.r + kRows - 1) / kRows, tiles = (v.c * a.grp + TILE - 1) / TILE;
  for (int blk = blockIdx.x * 8 + warp; blk < nblk; blk += gridDim.x * 8) {
    uint8_t* p = block_of(a.g, a.b.tables + (size_t)s * a.g.max_pages, a.layer, h, blk * kRows, nullptr);
    if (p == nullptr) continue;
    fetch<D>(smem_of(st), p, FEAT > 0, lane);
    cp_commit();
    cp_wait<0>();
    __syncwarp();
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    for (int tile = 0; tile < tiles; ++tile) {
      const int last = v.r - v.c + min(v.c - 1, (tile * TILE + TILE - 1) / a.grp), first = v.r - v.c + tile * TILE / a.grp;
      if (blk * kRows > last) continue;
      QTile<D, MODE> qt;
      load_q<D, MODE, FEAT>(qt, a, sq, s, h, tile, lane);
      float sc[P::NS][4][2];
      scores<D, MODE, FEAT>(qt, a, st, blk, (blk + 1) * kRows - 1 <= first, lane, sc);
#pragma unroll
      for (int ns = 0; ns < P::NS; ++ns)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = tile * TILE + column<MODE>(tig, ns, j), tok = row / a.grp, head = h * a.grp + row - tok * a.grp;
          if (tok >= v.c || (MODE == FP32_4 && tig >= 2)) continue;
          const float lse = a.lse[(size_t)(v.tok0 + tok) * a.g.nq + head];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] += ex2(sc[ns][i][j] - lse);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
    }
    if (tig == 0) {
      float* at = reinterpret_cast<float*>(p + weight_at(D)) + 4 * gid;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (blk * kRows + 4 * gid + i < v.r) at[i] += w[i];
    }
    __syncwarp();
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

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Dynamic shared memory at most: the SM's 227 KB less what each kernel declares statically.
constexpr int kAttnSmem = 225 * 1024, kSelectSmem = 208 * 1024;

// The dynamic shared memory limit of a kernel, raised once per device.
cudaError_t allow_smem(const void* fn, std::once_flag* once, int bytes) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  cudaError_t r = cudaSuccess;
  std::call_once(once[dev & 63], [&] { r = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
  return r;
}

template <typename... P, typename... Q>
cudaError_t launch(void (*fn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool overlap, Q... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&c, fn, args...);
}

// Units of the batch at most.
long long max_units(const Kv4Geom& g, const Kv4Batch& b, int tile) {
  const long long tiles = ((long long)b.max_count * (g.nq / g.nkv) + tile - 1) / tile;
  return (long long)b.n_seq * g.nkv * tiles * std::max(1, (b.max_rows + kRows - 1) / kRows);
}

template <int D, int MODE, int FEAT>
cudaError_t run_attention(AttnArgs a, int num_sms, cudaStream_t st) {
  constexpr int TILE = Shape<D, MODE>::TILE, kWarps = Shape<D, MODE>::kWarps, kStages = Shape<D, MODE>::kStages;
  a.warps = kWarps;
  using S = Stage<D>;
  static std::once_flag once[64], once_w[64];
  const size_t info = ((size_t)a.b.n_seq * sizeof(SeqInfo) + 127) / 128 * 128;
  const int dep_rows = std::min<long long>(TILE, (long long)a.b.max_count * a.grp);
  const size_t smem = info + (size_t)kWarps * kStages * S::kBytes + (size_t)kWarps * dep_rows * (D + 2) * 4;
  if (cudaError_t e = allow_smem((const void*)attn_kernel<D, MODE, FEAT>, once, kAttnSmem)) return e;
  const long long units = max_units(a.g, a.b, TILE);
  const int grid = (int)std::max<long long>(1, std::min<long long>(num_sms, (units + kWarps - 1) / kWarps));
  if (cudaError_t e = launch(attn_kernel<D, MODE, FEAT>, dim3(grid), kWarps * 32, smem, st, false, a)) return e;
  if (grid > 1) {
    const long long segs = (long long)a.g.nkv * (((long long)a.b.max_count * a.grp + TILE - 1) / TILE);
    if (cudaError_t e = launch(combine_kernel<D, TILE>, dim3((unsigned)std::min<long long>(segs, 4096), a.b.n_seq), 256, info, st, true, a)) return e;
  }
  if (a.lse != nullptr) {
    if (cudaError_t e = allow_smem((const void*)weight_kernel<D, MODE, FEAT>, once_w, kAttnSmem)) return e;
    const int bx = std::max(1, std::min(1024, (a.b.max_rows + 8 * kRows - 1) / (8 * kRows)));
    return launch(weight_kernel<D, MODE, FEAT>, dim3(bx, a.g.nkv, a.b.n_seq), 256, (size_t)8 * S::kBytes, st, false, a);
  }
  return cudaSuccess;
}

template <int D, int MODE>
cudaError_t pick_feat(const AttnArgs& a, int num_sms, cudaStream_t st) {
  if (a.b.max_count > 1 || a.a.window > 0) return run_attention<D, MODE, 2>(a, num_sms, st);
  if (a.a.cap > 0.f || a.a.slopes != nullptr) return run_attention<D, MODE, 1>(a, num_sms, st);
  return run_attention<D, MODE, 0>(a, num_sms, st);
}

// The narrowest tile that holds a sequence's queries of one KV head, or else the widest.
template <int D>
cudaError_t pick_attention(const AttnArgs& a, int num_sms, cudaStream_t st) {
  const long long cols = (long long)a.b.max_count * a.grp;
  if (a.a.bf16) return cols <= 8 ? pick_feat<D, BF16_8>(a, num_sms, st) : pick_feat<D, BF16_16>(a, num_sms, st);
  return cols <= 4 ? pick_feat<D, FP32_4>(a, num_sms, st) : pick_feat<D, FP32_8>(a, num_sms, st);
}

// Tokens of a CTA of append and read: about 2,048 vectors of 8.
int tokens_per_cta(const Kv4Geom& g) { return std::max(1, 2048 / (g.nkv * 2 * (g.d / 8))); }

}  // namespace

size_t kv4_attention_workspace(const Kv4Geom& g, const Kv4Batch& b, int num_sms) {
  return round256((size_t)num_sms * 2 * 16 * (g.d + 2) * 4) + round256((size_t)b.n_tokens * g.nq * 4);
}

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

cudaError_t kv4_attention(const Kv4Geom& g, int layer, const Kv4Batch& b, const Kv4Attn& at, void* ws, int num_sms, cudaStream_t st) {
  AttnArgs a;
  a.g = g;
  a.b = b;
  a.a = at;
  a.layer = layer;
  a.grp = g.nq / g.nkv;
  a.grid_max = num_sms;
  a.cap2 = at.cap > 0.f ? 2.f * kLog2e / at.cap : 0.f;
  a.part = reinterpret_cast<float*>(ws);
  a.lse = at.accumulate ? reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + round256((size_t)num_sms * 2 * 16 * (g.d + 2) * 4)) : nullptr;
  return g.d == 64 ? pick_attention<64>(a, num_sms, st) : pick_attention<128>(a, num_sms, st);
}

cudaError_t kv4_evict(const Kv4Geom& g, int layer0, int n_layers, int n_seq, int max_rows, const int32_t* rows,
                      const int32_t* tables, const int32_t* next_pos, int keep, int recent, const int32_t* out_tables,
                      int out_pages, int32_t* rows_out, int32_t* status, void* ws, cudaStream_t st) {
  static std::once_flag once[2][64];
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
