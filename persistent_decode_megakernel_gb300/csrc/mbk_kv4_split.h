// mbk_kv4_split.h -- what the two attention kernels share: a sequence's share of the work, the join of partial
// results and the output's type.  Included by the .cu files only.
#pragma once
#include "mbk_kv4_device.h"

namespace mbk {
namespace {

struct SeqInfo {
  int cum, r, c, tok0;  // units of work before the sequence; rows, new tokens, first token
};

constexpr int kMinRun = 8;  // key tiles of a run at least, where a prompt's keys are split

// Division of query rows by the group's heads, by multiplication: exact below 2^28 rows and 17 heads.
struct ByGroup {
  unsigned inverse;  // ceil(2^32 / heads), 0 for one head
  __host__ __device__ static ByGroup of(int heads) { return ByGroup{heads == 1 ? 0u : (unsigned)(((1ull << 32) + heads - 1) / heads)}; }
};
__device__ __forceinline__ int operator/(int row, ByGroup d) { return d.inverse == 0u ? row : (int)__umulhi((unsigned)row, d.inverse); }

struct PromptArgs {
  Kv4Geom g;
  Kv4Batch b;
  Kv4Attn a;
  int layer, grp;
  ByGroup by_grp;
  int least;     // query rows per KV head from which on a sequence is this kernel's
  int slots;     // CTAs that the GPU holds
  float scale2, cap_in, cap_out;  // scale log2(e); 2 / cap, cap log2(e)
  float* part;   // [item][128][d + 4]
  float* lse;    // [n_tokens][nq] log2 of the softmax denominators, or null
};

// Exclusive scan over the block (sums: one int per warp) and its total; all threads call.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__device__ __forceinline__ void store_out(const Kv4Attn& a, size_t at, const float (&x)[8]) {
  if (a.bf16) store8(reinterpret_cast<__nv_bfloat16*>(a.out) + at, x);
  else store8(reinterpret_cast<float*>(a.out) + at, x);
}

// Writes eight dims of a column: the output and (first dims) lse, or with `to` a joined partial.
template <int D, typename Args>
__device__ __forceinline__ void store_joined(const Args& a, const SeqInfo& sq, int h, int row0, int col, int d0, float* to, float m, float l,
                                             float (&o)[8]) {
  constexpr int kPart = D + 4;
  if (to != nullptr) {
    store8(to + col * kPart + d0, o);
    if (d0 == 0) {
      to[col * kPart + D] = m;
      to[col * kPart + D + 1] = l;
    }
  } else {
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= inv;
    const int row = row0 + col, tok = row / a.by_grp, head = h * a.grp + row - tok * a.grp;
    store_out(a.a, (size_t)(sq.tok0 + tok) * a.a.ldo + (size_t)head * D + d0, o);
    if (a.lse != nullptr && d0 == 0) a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] = l > 0.f ? m + log2f(l) : INFINITY;
  }
}
// Adds partial p's share of eight dims, relative to `base`.
template <int D>
__device__ __forceinline__ void add_partial(const float* p, int d0, float base, float& l, float (&o)[8]) {
  const float w = ex2(p[D] - base);
  const float4 u = *reinterpret_cast<const float4*>(p + d0), v = *reinterpret_cast<const float4*>(p + d0 + 4);
  l = fmaf(p[D + 1], w, l);
  o[0] = fmaf(u.x, w, o[0]), o[1] = fmaf(u.y, w, o[1]), o[2] = fmaf(u.z, w, o[2]), o[3] = fmaf(u.w, w, o[3]);
  o[4] = fmaf(v.x, w, o[4]), o[5] = fmaf(v.y, w, o[5]), o[6] = fmaf(v.z, w, o[6]), o[7] = fmaf(v.w, w, o[7]);
}

// One warp joins n partials of one column, at(k) being the k-th's place: a lane takes eight dims of every 4th (d 128:
// every 2nd) partial.
template <int D, typename Args, typename At>
__device__ __forceinline__ void join_column(const Args& a, const SeqInfo& sq, int h, int row0, int col, int n, float* to, At at) {
  constexpr int kPart = D + 4, kChunks = D / 8;
  const int lane = threadIdx.x & 31, d0 = lane % kChunks * 8;
  float m = -INFINITY;
  for (int k = 0; k < n; ++k) m = fmaxf(m, at(k)[col * kPart + D]);
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int k = lane / kChunks; k < n; k += 32 / kChunks) add_partial<D>(at(k) + col * kPart, d0, base, l, o);
#pragma unroll
  for (int i = kChunks; i < 32; i <<= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, i);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], i);
  }
  if (lane < kChunks) store_joined<D>(a, sq, h, row0, col, d0, to, m, l, o);
}

// Joins n partials of a segment of `cols` columns, at(k) being the k-th's place, and writes the output (and
// lse), or with `to` the joined partial.  2^x threads take the partials of 8 dims of a column between them.  All
// threads of the CTA call.
template <int D, typename Args, typename At>
__device__ __forceinline__ void join(const Args& a, const SeqInfo& sq, int h, int row0, int cols, int n, float* to, At at) {
  constexpr int kPart = D + 4;
  const int items = cols * (D / 8);
  int sl = 32;
  while (sl > 1 && (sl >= 2 * n || items * sl > (int)blockDim.x)) sl >>= 1;
  for (int x = threadIdx.x; x < (items * sl + 31) / 32 * 32; x += blockDim.x) {
    const int item = min(x / sl, items - 1), k0 = x % sl, col = item / (D / 8), d0 = item % (D / 8) * 8;
    float m = -INFINITY;
#pragma unroll 4
    for (int k = k0; k < n; k += sl) m = fmaxf(m, at(k)[col * kPart + D]);
    for (int i = 1; i < sl; i <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, i));
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = k0; k < n; k += sl) add_partial<D>(at(k) + col * kPart, d0, base, l, o);
    for (int i = 1; i < sl; i <<= 1) {
      l += __shfl_xor_sync(0xffffffffu, l, i);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], i);
    }
    if (k0 == 0 && x / sl < items) store_joined<D>(a, sq, h, row0, col, d0, to, m, l, o);
  }
}

}  // namespace
}  // namespace mbk
