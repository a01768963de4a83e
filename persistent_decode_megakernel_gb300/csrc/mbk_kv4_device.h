// mbk_kv4_device.h -- what the 4-bit KV cache's kernels share: bounds-checked views of a batch and its pages,
// vector loads, codes as tensor-core operands, launches.  Included by the .cu files only.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "mbk_kv4.h"

namespace mbk {
namespace {

constexpr int kRows = kKv4Rows;
constexpr float kLog2e = 1.4426950408889634f;

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

// ------------------------------------------------------------------ vectors of 8 elements
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
// ------------------------------------------------------------------ copies and matrix instructions
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
// (a, b) += s (c, d) in one instruction.
__device__ __forceinline__ void add2(float& a, float& b, float c, float d, float s) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n mov.b64 z, {%4, %4};\n fma.rn.f32x2 x, y, z, x;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b) : "f"(c), "f"(d), "f"(s));
}
// (a, b) += (c, d) in one instruction.
__device__ __forceinline__ void add2(float& a, float& b, float c, float d) {
  asm("{\n .reg .b64 x, y;\n mov.b64 x, {%0, %1};\n mov.b64 y, {%2, %3};\n add.rn.f32x2 x, x, y;\n mov.b64 {%0, %1}, x;\n}\n"
      : "+f"(a), "+f"(b) : "f"(c), "f"(d));
}
// The codes of a word as four operand registers (codes i and i + 4 in register i), in units of
// 2^-24 (16 times that in registers 1 and 3), with PRECISE of 2^-18.  flip (PRECISE): 0, or all ones for 15 - code.
template <bool PRECISE>
__device__ __forceinline__ void codes(uint32_t x, uint32_t (&r)[4], uint32_t flip = 0u) {
  constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kTop = 0x03c003c0u;
  if (PRECISE) {
    r[0] = ((x << 6) ^ flip) & kTop;
    r[1] = ((x << 2) ^ flip) & kTop;
    r[2] = ((x >> 2) ^ flip) & kTop;
    r[3] = ((x >> 6) ^ flip) & kTop;
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
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Two fp32 values in a register pair, and the instructions on both at once.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair_of(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 halves(f2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 sum2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// ------------------------------------------------------------------ launches
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// The dynamic shared memory limit of a kernel, raised once per device.
cudaError_t allow_smem(const void* fn, std::atomic<bool>* done, int bytes) {
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (done[dev & 63].load(std::memory_order_relaxed)) return cudaSuccess;
  if (cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  done[dev & 63].store(true, std::memory_order_relaxed);
  return cudaSuccess;
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

}  // namespace
}  // namespace mbk
