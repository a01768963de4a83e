// mbk_kv4.h -- the 4-bit KV cache's pool, batches and launches (mbk_kv4_attn.cu,
// mbk_kv4_rows.cu), used by the C ABI
// (mbk_kv4_api.cu) and by the prefill path of a handle whose pool is held in 4 bits.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mbk.h"

namespace mbk {

constexpr int kKv4Rows = 32;      // rows of a block of the pool
constexpr int kKv4Group = 64;     // elements that share a (scale, lo) pair
constexpr int kKv4MaxSeqs = MBK_KV4_MAX_SEQS;
constexpr int kKv4MaxGroup = 16;  // query heads per KV head, as everywhere in the library

// The pool as the kernels address it: block b of page g for (layer, head) starts at
// pool + g * page_stride + ((layer * nkv + head) * blocks_per_page + b) * block_bytes.
struct Kv4Geom {
  uint8_t* pool;
  unsigned long long page_stride;
  unsigned head_stride;  // bytes of one (page, layer, head)
  int num_pages, L, nq, nkv, d, track;
  int page_shift;        // log2 of the page size in rows
  int max_pages;         // entries of a sequence's page table
  int block_bytes;
};

struct Kv4Batch {
  int n_seq, n_tokens, max_count, max_rows;
  const int32_t* offsets;    // [n_seq + 1] tokens of sequence s: [offsets[s], offsets[s + 1])
  const int32_t* rows;       // [n_seq] rows of the sequence, the new tokens' included
  const int32_t* positions;  // [n_seq] position of the sequence's first new token, or null: its row
  const int32_t* tables;     // [n_seq][max_pages]
  int32_t* status;           // device word that errors are OR-ed into, or null
};

struct Kv4Attn {
  const void* q;
  void* out;
  long long ldq, ldo;        // elements between tokens
  int bf16;                  // q and out: bf16 instead of fp32
  float scale, cap;
  const float* slopes;       // [nq] or null
  int window;                // 0: none
  int accumulate;
};

// Bytes that a call's workspace needs (0 is possible); the arguments are checked by the caller.
size_t kv4_attention_workspace(const Kv4Geom& g, const Kv4Batch& b, int num_sms);
size_t kv4_evict_workspace(const Kv4Geom& g, int n_layers, int n_seq, int keep);

cudaError_t kv4_append(const Kv4Geom& g, int layer, const Kv4Batch& b, const void* k, const void* v, long long ld, int bf16,
                       cudaStream_t st);
cudaError_t kv4_read(const Kv4Geom& g, int layer, const Kv4Batch& b, void* k, void* v, long long ld, int bf16, cudaStream_t st);
cudaError_t kv4_attention(const Kv4Geom& g, int layer, const Kv4Batch& b, Kv4Attn a, void* ws, int num_sms, cudaStream_t st);
// The prompt kernel: the batch's sequences of at least `least` query rows per KV head (bf16, or fp32 with d 64).  part:
// kv4_prompt_partials bytes; lse: [n_tokens][nq] or null.
size_t kv4_prompt_partials(const Kv4Geom& g, const Kv4Batch& b, int num_sms);
cudaError_t kv4_prompt(const Kv4Geom& g, int layer, const Kv4Batch& b, const Kv4Attn& a, int least, float* part, float* lse, int num_sms,
                       cudaStream_t st);
cudaError_t kv4_evict(const Kv4Geom& g, int layer0, int n_layers, int n_seq, int max_rows, const int32_t* rows,
                      const int32_t* tables, const int32_t* next_pos, int keep, int recent, const int32_t* out_tables,
                      int out_pages, int32_t* rows_out, int32_t* status, void* ws, int num_sms, cudaStream_t st);

// MBK_OK, or MBK_ERR_INVALID_ARG for a configuration that the kernels do not take.
int kv4_config_check(const mbk_kv4_config* c);
Kv4Geom kv4_geom(const mbk_kv4_config& c, void* pool);

}  // namespace mbk
