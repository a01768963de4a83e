// mbk_kv4_prompt.cu -- attention of many query rows (prompts, chunks of prompts) over the 4-bit KV cache, on
// tcgen05.
//
// A CTA takes 256 query rows -- (token, query head) pairs that read one KV head -- as two tiles of 128 through a run
// of key tiles of 64 cache rows.  Four warps turn K's rows into fp16 operands in shared memory (128-byte
// swizzle, [row][dim]) and four V's ([dim][row]), once for both query tiles; a lane of the first issues the matrix
// instructions in between; and a thread of the other eight warps owns a query row: it reads the row's scores from
// tensor memory, keeps its softmax and writes its weights over the scores, where the second product takes them
// from.  Scores have two buffers and K and V two stages, so that conversion and tensor cores work one tile
// ahead of the softmax.  (Two CTAs of one query tile and four conversion warps each were slower, 400 us where this form
// then took 246: the conversion held the softmax up.)
//   bf16: K and V are the values lo + scale * code rounded to fp16 (one rounding, 2^-11; bf16 has 2^-8),
// the weights are rounded to fp16 too.
//   fp32 (head dim 64): the operands are code - 8, exact; q and the weights are hi + lo fp16 (22 bits); the
// softmax applies the rows' scale and lo, as the decode kernel does.  The tensor cores' sums are truncated, so the
// output is moved to a second buffer and added there in fp32 every 2 tiles; and as the truncation leaves a bias in each such
// group (which reached 3.6e-5 of the output at 130,000 rows), every other group takes 15 - code and is subtracted.
//   Bound by the softmax, which therefore goes two values at a time where the GPU has a form for it: of some 4,600 clocks a
// key tile (both query tiles) 1,300 are scale and maximum and 2,500 exponentials, split and store, two warps a scheduler
// that wait for their own results (issue slots 39% busy, tensor cores 16%).  Measured: the last 2,048 tokens of 8,192 rows,
// 9 and 3 heads, d 64, fp32: 228 us with the join, 148 TFLOP/s of the formula's; four prompts of up to 1,024 tokens over up
// to 4,096 rows, 32 and 8 heads, d 128, bf16, cap and window: 363 us.
#include "mbk_kv4_device.h"
#include "mbk_kv4_split.h"

namespace mbk {
namespace {

constexpr int kQ = 128;        // query rows of a tile: tensor-memory lanes
constexpr int kItem = 256;     // query rows of an item: two tiles
constexpr int kKeys = 64;      // cache rows of a key tile: one 128-byte row of fp16
constexpr int kThreads = 512;  // softmax 2 x 128, K 128, V 128
constexpr int kTmemCols = 512; // per query tile: scores 2 x 64, output 64 or 128, fp32: sums 64
// fp32: tiles between two moves of the output.  Measured at 20,000 rows, queries of 0.3 (fp32 arithmetic itself: 5.5e-7 off):
// every 8 2.0e-6 off, 4 9e-7, 2 5.4e-7; the last 2,048 tokens of 8,192 rows in 217, 222 and 231 us.
constexpr int kFlush = 2;
// fp32: every other such group takes V's codes from above (15 - code) and is subtracted, see the top.
__device__ __forceinline__ bool odd_group(int j) { return j / kFlush & 1; }
constexpr int kMaxRounds = 4;  // items per CTA at most, about, where keys are split
constexpr int kNotes = 4;      // tiles whose notes and pairs are kept
constexpr float kSlack = 8.f;  // a running maximum is renewed when a score exceeds it by 2^8
constexpr unsigned long long kWaitNs = 2000000000ull;

// tcgen05.mma kind::f16: fp32 sums (bits 4-5 = 1), both operands fp16 (bits 7-12 = 0) and K-major,
// N / 8 in bits 17-22, M / 16 in bits 24-28.
__device__ constexpr uint32_t idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kQ >> 4) << 24); }

__device__ __forceinline__ void mbar_init(uint64_t* b, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_of(b)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* b, unsigned parity) {
  unsigned ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_of(b)), "r"(parity)
               : "memory");
  return ok != 0;
}
// Waits for the phase of the given parity; false after kWaitNs, or once another thread has given up.
__device__ __forceinline__ bool mbar_wait_slow(uint64_t* b, unsigned parity, volatile unsigned* failed) {
  unsigned long long t0 = 0ull;
  for (unsigned spins = 0;; ++spins) {
    if (mbar_test(b, parity)) return true;
    if ((spins & 63u) == 63u) {
      if (*failed != 0u) return false;
      unsigned long long t;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (t0 == 0ull) t0 = t;
      else if (t - t0 > kWaitNs) {
        *failed = 1u;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint64_t* b, unsigned parity, volatile unsigned* failed) {
  return mbar_test(b, parity) || mbar_wait_slow(b, parity, failed);
}
// The same for a whole warp, which goes on or gives up together.
__device__ __forceinline__ bool warp_wait(uint64_t* b, unsigned parity, volatile unsigned* failed) {
  return __all_sync(0xffffffffu, mbar_wait(b, parity, failed));
}

// A K-major operand tile with the 128-byte swizzle: rows of 64 fp16 (128 bytes), 8 rows a group of 1024
// bytes; a step of 16 along K moves the start by 32 bytes.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ void umma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a),
               "l"(b), "r"(desc), "r"(accumulate)
               : "memory");
}
// The same with the first operand in tensor memory: a row a lane, two fp16 a column.
__device__ __forceinline__ void umma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, uint32_t accumulate) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a),
               "l"(b), "r"(desc), "r"(accumulate)
               : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_of(bar)) : "memory");
}
// One lane of a converged warp, always the same one.  The matrix instructions take their operands from uniform registers;
// in a branch on a thread index the compiler would move each of them there, one by one (85 clocks an instruction).
__device__ __forceinline__ bool elected() {
  unsigned p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0u;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t at, f2* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(at));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = pair_of(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]),
      "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
      "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])),
      "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])),
      "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int N>
struct Const {
  static constexpr int value = N;
};

// The shared memory of a CTA.
template <int D, bool FP32>
struct Layout {
  static constexpr int kGroups = D / 64, kHalves = FP32 ? 2 : 1;
  static constexpr int kQTile = kQ * 128 * kGroups * kHalves;   // per half and group: [128][64] fp16
  static constexpr int kQBytes = 2 * kQTile;
  static constexpr int kTile = kKeys * 128 * kGroups;           // K: per group [64 rows][64 dims]; V: [D dims][64 rows]
  static constexpr int kQAt = 0, kKAt = kQBytes, kVAt = kKAt + 2 * kTile;
  static constexpr int kPairsAt = kVAt + 2 * kTile;             // fp32: float [kNotes][4: sk, zk, sv, zv][64]
  static constexpr int kPosAt = kPairsAt + (FP32 ? kNotes * kKeys * 16 : 0);
  static constexpr int kInfoAt = kPosAt + kNotes * kKeys * 4;   // then SeqInfo [n_seq]
};

// What the conversion tells the softmax about a tile.  Written with K, at most two tiles ahead of the scores, which are
// one ahead of the softmax: four slots.
struct TileNote {
  unsigned bad;        // bit b: block b of the tile lies in a page outside the pool
  int e[2];            // fp32: exponent of the largest scale of V, per 32 rows
  unsigned nan[2][2];  // rows whose V is NaN, per group of 64 dims and 32 rows (they are zero for the products)
};

// ---------------------------------------------------------------- work items
// An item is (sequence, KV head, 256 query rows, run of at most kt key tiles).  Items go round the CTAs, the
// tiles with most keys first.
struct Work {
  int n_seq, nkv, grp, window, track, kt, total;
  const SeqInfo* seq;
  __device__ int tiles(const SeqInfo& q) const { return (q.c * grp + kItem - 1) / kItem; }
  __device__ int first_of(const SeqInfo& q, int tile) const {
    return window > 0 && !track ? max(0, q.r - q.c + tile * kItem / grp - window + 1) / kKeys : 0;
  }
  __device__ int end_of(const SeqInfo& q, int tile) const {  // key tiles [first, end) of a query tile
    const int last = q.r - q.c + min(q.c - 1, (tile * kItem + kItem - 1) / grp);
    return last < 0 ? 0 : last / kKeys + 1;
  }
  __device__ int span(const SeqInfo& q) const {  // key tiles of a query tile at most
    int n = max(1, (q.r + kKeys - 1) / kKeys);
    if (window > 0 && !track) n = min(n, (window + kItem / grp + 1) / kKeys + 2);
    return n;
  }
  __device__ int splits(const SeqInfo& q) const { return (span(q) + kt - 1) / kt; }
  __device__ int parts(const SeqInfo& q, int tile) const {  // the splits of a query tile that have keys
    return (max(0, end_of(q, tile) - first_of(q, tile)) + kt - 1) / kt;
  }
};
struct Item {
  int s, h, tile, split, k0, k1, parts;
};
__device__ __forceinline__ Item item_at(const Work& w, int i) {
  int lo = 0, hi = w.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (w.seq[mid].cum <= i) lo = mid; else hi = mid - 1;
  }
  const SeqInfo q = w.seq[lo];
  Item it;
  it.s = lo;
  int rem = i - q.cum;
  it.h = rem % w.nkv;
  rem /= w.nkv;
  const int ns = w.splits(q);
  it.split = rem % ns;
  it.tile = w.tiles(q) - 1 - rem / ns;
  it.parts = w.parts(q, it.tile);
  it.k0 = w.first_of(q, it.tile) + it.split * w.kt;
  it.k1 = min(it.k0 + w.kt, w.end_of(q, it.tile));
  return it;
}

// Fills info and returns the work; all threads call.  Two passes: units first, to choose the runs' length, then items.
__device__ Work make_work(const PromptArgs& a, SeqInfo* info, int* sums, bool report) {
  Work w;
  w.n_seq = a.b.n_seq;
  w.nkv = a.g.nkv;
  w.grp = a.grp;
  w.window = a.a.window;
  w.track = a.g.track;
  w.seq = info;
  w.kt = 1 << 28;
  long long units = 0, segs = 0;
  int carry = 0;
  for (int pass = 0; pass < 2; ++pass) {
    carry = 0;
    for (int s0 = 0; s0 < a.b.n_seq; s0 += blockDim.x) {
      const int s = s0 + threadIdx.x;
      SeqInfo q{0, 0, 0, 0};
      if (s < a.b.n_seq) {
        const SeqView v = seq_view(a.g, a.b, s, report && pass == 0);
        q.r = v.r;
        q.c = v.c * a.grp >= a.least ? v.c : 0;  // shorter ones are the decode kernel's
        q.tok0 = v.tok0;
      }
      const int n = q.c == 0 ? 0 : w.tiles(q) * w.nkv * (pass == 0 ? w.span(q) : w.splits(q));
      int total;
      q.cum = carry + block_scan(n, sums, &total);
      if (s < a.b.n_seq) info[s] = q;
      carry += total;
      if (pass == 0) {
        block_scan(q.c == 0 ? 0 : w.tiles(q) * w.nkv, sums, &total);
        segs += total;
      }
    }
    if (pass == 0) {
      units = carry;
      // Split along the keys only when whole query tiles would not fill the GPU twice, into runs of the length
      // that ends first: rounds of items on all slots, each run costing its tiles and about 3 more.
      if (segs < 2ll * a.slots) {
        long long best = -1;
        int run = 0;
        for (int rounds = 1; rounds <= kMaxRounds; ++rounds) {
          w.kt = max(kMinRun, (int)((units + (long long)rounds * a.slots - 1) / ((long long)rounds * a.slots)));
          int items = 0;
          for (int s0 = 0; s0 < a.b.n_seq; s0 += blockDim.x) {
            const int s = s0 + threadIdx.x;
            const SeqInfo q = s < a.b.n_seq ? info[s] : SeqInfo{0, 0, 0, 0};
            int total;
            block_scan(q.c == 0 ? 0 : w.tiles(q) * w.nkv * w.splits(q), sums, &total);
            items += total;
          }
          const long long cost = (long long)((items + a.slots - 1) / a.slots) * (w.kt + 3);
          if (best < 0 || cost < best) {
            best = cost;
            run = w.kt;
          }
          if (w.kt == kMinRun) break;
        }
        w.kt = run;
      }
    }
    __syncthreads();
  }
  w.total = carry;
  return w;
}

// ---------------------------------------------------------------- conversion: 64 rows of K or V to operands
// Loads that stay where they are written: the compiler would move plain ones down to their use, a tile later.
__device__ __forceinline__ uint32_t load_now(const uint32_t* p) {
  uint32_t r;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}
__device__ __forceinline__ uint4 load_now(const uint4* p) {
  uint4 r;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t as_word(__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); }

// The codes i and i + 4 of a word (or, of a permuted word, of two rows), as fp16 less 8 (CENTRE) or as they are.
template <bool CENTRE>
__device__ __forceinline__ void code_pairs(uint32_t x, __half2 (&r)[4]) {
  constexpr float c = CENTRE ? 8.f : 0.f;
  const __half2 low = __float2half2_rn(-1024.f - c), high = __float2half2_rn(-64.f - c), frac = __float2half2_rn(0.0625f);
  const uint32_t x8 = x >> 8;
  r[0] = __hadd2(as_half2((x & 0x000f000fu) | 0x64006400u), low);           // 1024 + code
  r[1] = __hfma2(as_half2((x & 0x00f000f0u) | 0x64006400u), frac, high);    // 1024 + 16 code
  r[2] = __hadd2(as_half2((x8 & 0x000f000fu) | 0x64006400u), low);
  r[3] = __hfma2(as_half2((x8 & 0x00f000f0u) | 0x64006400u), frac, high);
}

// fp16 (scale, lo) with lo + 15 scale within fp16: a scale that was rounded up may lead beyond, at the type's very end.
__device__ __forceinline__ uint32_t within(uint32_t pair) {
  if ((pair & 0x7fffu) < 0x6800u && (pair >> 16 & 0x7fffu) < 0x7800u) return pair;  // below 2^11 and 2^15: far from it
  const float2 p = unpack_half(pair);
  if (!(fmaf(15.f, p.x, p.y) >= 65520.f)) return pair;
  return (pair & 0xffff0000u) | __half_as_ushort(__float2half_rd((65504.f - p.y) / 15.f));
}

// What a thread (t of 128) of the K warps holds of a tile before it converts it: 32 dims of row t / 2 per group, and
// for the notes V's pair of row t % 64, group t / 64.
template <int D>
struct RawK {
  static constexpr int kGroups = D / 64;
  uint4 k[kGroups];
  uint32_t kp[kGroups], vp;
  int pos;
  unsigned bad;
  __device__ __forceinline__ void load(const PromptArgs& a, const uint8_t* b0, const uint8_t* b1, int t) {
    bad = (b0 == nullptr ? 1u : 0u) | (b1 == nullptr ? 2u : 0u);
    const uint8_t* kb = t < 64 ? b0 : b1;
    const int kr = (t >> 1) & 31;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      k[g] = make_uint4(0u, 0u, 0u, 0u);
      kp[g] = 0u;
      if (kb != nullptr) {
        k[g] = load_now(reinterpret_cast<const uint4*>(kb + kr * (D / 2) + g * 32 + (t & 1) * 16));
        kp[g] = load_now(reinterpret_cast<const uint32_t*>(kb + code_bytes(D) + (kr * kGroups + g) * 4));
      }
    }
    pos = 0;
    if (a.g.track && (t & 1) == 0 && kb != nullptr) pos = (int)load_now(reinterpret_cast<const uint32_t*>(kb + pos_at(D) + 4 * kr));
    const uint8_t* vb = (t & 32) ? b1 : b0;
    vp = 0u;
    if (vb != nullptr && (t >> 6) < kGroups)
      vp = load_now(reinterpret_cast<const uint32_t*>(vb + half_bytes(D) + code_bytes(D) + ((t & 31) * kGroups + (t >> 6)) * 4));
  }
};
// ... and of the V warps: of rows 4 (t % 16) .. + 3 the word t / 16 (8 dims) per group.
template <int D>
struct RawV {
  static constexpr int kGroups = D / 64;
  uint32_t v[kGroups][4], vp[kGroups][4];
  __device__ __forceinline__ void load(const PromptArgs& a, const uint8_t* b0, const uint8_t* b1, int t) {
    const uint8_t* vb = (t & 15) < 8 ? b0 : b1;
    const int vr = 4 * (t & 7), vw = t >> 4;
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[g][i] = vp[g][i] = 0u;
        if (vb != nullptr) {
          v[g][i] = load_now(reinterpret_cast<const uint32_t*>(vb + half_bytes(D) + (vr + i) * (D / 2) + g * 32 + vw * 4));
          vp[g][i] = load_now(reinterpret_cast<const uint32_t*>(vb + half_bytes(D) + code_bytes(D) + ((vr + i) * kGroups + g) * 4));
        }
      }
  }
};

// K of a tile to its stage, and what the softmax has to know: positions, bad pages, V's NaN rows, fp32: the pairs.
template <int D, bool FP32>
__device__ __forceinline__ void convert_k(const RawK<D>& w, const PromptArgs& a, unsigned char* kst, unsigned char* smem, int slot, int row0,
                                          int rows, int t, bool odd, TileNote* note) {
  using L = Layout<D, FP32>;
  constexpr int kGroups = D / 64;
  const int key = t >> 1, half = t & 1;
  const bool kon = row0 + key < rows, von = row0 + (t & 63) < rows;
  const unsigned nan = __ballot_sync(0xffffffffu, von && (w.vp & 0x7fffu) > 0x7c00u);
  const uint32_t vp = von && (w.vp & 0x7fffu) <= 0x7c00u ? w.vp : 0u;
  if ((t & 31) == 0) note->nan[t >> 6][(t >> 5) & 1] = nan;
  if (t == 0) note->bad = w.bad;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    // four chunks of 8 dims, in the order 0 4 1 5 2 6 3 7 (q is stored in the same order)
    unsigned char* kt = kst + g * kKeys * 128 + key * 128;
    const uint32_t words[4] = {w.k[g].x, w.k[g].y, w.k[g].z, w.k[g].w};
    const __half2 p = as_half2(kon ? within(w.kp[g]) : 0u), s2 = __low2half2(p), z2 = __high2half2(p);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      __half2 r[4];
      code_pairs<FP32>(words[c], r);
      uint4 o;
      if (FP32) o = make_uint4(as_word(r[0]), as_word(r[1]), as_word(r[2]), as_word(r[3]));
      else o = make_uint4(as_word(__hfma2(r[0], s2, z2)), as_word(__hfma2(r[1], s2, z2)), as_word(__hfma2(r[2], s2, z2)), as_word(__hfma2(r[3], s2, z2)));
      *reinterpret_cast<uint4*>(kt + (((4 * half + c) ^ (key & 7)) << 4)) = o;
    }
  }
  if (FP32) {
    // the rows' pairs, lo moved to the codes' middle (odd groups count 7 - code), and V's largest scale
    float* pairs = reinterpret_cast<float*>(smem + L::kPairsAt) + slot * 4 * kKeys;
    if (half == 0) {
      const float2 p = unpack_half(kon ? w.kp[0] : 0u);
      pairs[key] = p.x;
      pairs[kKeys + key] = fmaf(8.f, p.x, p.y);
    }
    if (t < 64) {
      const float2 p = unpack_half(vp);
      pairs[2 * kKeys + t] = p.x;
      pairs[3 * kKeys + t] = fmaf(odd ? 7.f : 8.f, p.x, p.y);
      const unsigned e = __reduce_max_sync(0xffffffffu, (vp >> 10) & 31u);
      if ((t & 31) == 0) note->e[t >> 5] = min((int)e - 15, 15);
    }
  }
  if (a.g.track && half == 0) reinterpret_cast<int*>(smem + L::kPosAt)[slot * kKeys + key] = w.pos;
}

// V of a tile to its stage, transposed: of rows vk .. vk + 3, 8 bytes of each of 8 dims' rows.  flip (fp32): 0, or all
// ones for 15 - code.
template <int D, bool FP32>
__device__ __forceinline__ void convert_v(const RawV<D>& w, unsigned char* vst, int row0, int rows, int t, uint32_t flip) {
  constexpr int kGroups = D / 64;
  const int vk = 4 * (t & 15), vw = t >> 4;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    unsigned char* vt = vst + (g * 64 + vw * 8) * 128;
    __half2 s01{}, s23{}, z01{}, z23{};
    if (!FP32) {
      uint32_t vp[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)  // rows behind the end, and NaN groups (which the softmax is told of), are zeros
        vp[i] = row0 + vk + i < rows && (w.vp[g][i] & 0x7fffu) <= 0x7c00u ? within(w.vp[g][i]) : 0u;
      s01 = as_half2(__byte_perm(vp[0], vp[1], 0x5410));
      z01 = as_half2(__byte_perm(vp[0], vp[1], 0x7632));
      s23 = as_half2(__byte_perm(vp[2], vp[3], 0x5410));
      z23 = as_half2(__byte_perm(vp[2], vp[3], 0x7632));
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t sel = hf ? 0x7632u : 0x5410u;
      __half2 x[4], y[4];
      code_pairs<FP32>(__byte_perm(w.v[g][0], w.v[g][1], sel) ^ flip, x);
      code_pairs<FP32>(__byte_perm(w.v[g][2], w.v[g][3], sel) ^ flip, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int dim = 4 * hf + j;  // row of the tile: g * 64 + 8 vw + dim; its low three bits are dim
        uint2 o;
        if (FP32) o = make_uint2(as_word(x[j]), as_word(y[j]));
        else o = make_uint2(as_word(__hfma2(x[j], s01, z01)), as_word(__hfma2(y[j], s23, z23)));
        *reinterpret_cast<uint2*>(vt + dim * 128 + (((vk >> 3) ^ dim) << 4) + (vk & 4) * 2) = o;
      }
    }
  }
}

// ---------------------------------------------------------------- the kernel
template <int D, bool FP32, bool FEAT>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptArgs a) {
  using L = Layout<D, FP32>;
  constexpr int kGroups = D / 64;
  extern __shared__ unsigned char raw_smem[];
  __shared__ __align__(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2][2], pv_done[2][2], p_full[2][2], q_full, drain;  // [query tile][stage]
  __shared__ uint32_t tmem_slot;
  __shared__ unsigned failed;
  __shared__ TileNote notes[kNotes];
  __shared__ int sums[kThreads / 32];
  __shared__ float2 row_scale[kItem];
  unsigned char* smem = raw_smem + ((1024u - (smem_of(raw_smem) & 1023u)) & 1023u);
  SeqInfo* info = reinterpret_cast<SeqInfo*>(smem + L::kInfoAt);
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 128);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 128);
      mbar_init(&v_empty[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&s_full[h][i], 2);
        mbar_init(&pv_done[h][i], 1);
        mbar_init(&p_full[h][i], 128);
      }
    }
    mbar_init(&q_full, 256);
    mbar_init(&drain, 1);
    failed = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 15) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&tmem_slot)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const Work work = make_work(a, info, sums, blockIdx.x == 0);
  fence_before();
  __syncthreads();
  fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = tmem_slot;
  volatile unsigned* abort = &failed;
  unsigned tile_no = 0;  // key tiles so far: every role counts them alike

  if (warp >= 8) {
    // ------------------------------------------------------------ conversion (warps 8, 9, 12, 13: K, the others: V) and matrix instructions
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");  // of 128 at launch; the softmax takes them
    // two warps of one kind on a scheduler (warp % 4), not one of each: it then has less code to fetch
    const bool for_k = (warp & 2) == 0;
    const int t = (warp >= 12 ? 64 : 0) + (warp & 1) * 32 + (threadIdx.x & 31);
    bool ok = true;
    // descriptors of the operands' first tiles; 16 bytes on are 1 more
    const uint64_t q_desc = tile_desc(smem_of(smem + L::kQAt)), k_desc = tile_desc(smem_of(smem + L::kKAt)), v_desc = tile_desc(smem_of(smem + L::kVAt));
    unsigned items = 0;
    // (warp 8) S = Q K^T of key tile number `no`, the item's j-th, for both query tiles; ST: the tile's stage
    auto score_at = [&](auto ST) {
      constexpr int st = decltype(ST)::value;
      if (elected()) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int hf = 0; hf < L::kHalves; ++hf)
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma(tmem + h * 256 + st * kKeys, q_desc + h * (L::kQTile / 16) + (hf * kGroups + g) * (kQ * 8) + ks * 2,
                     k_desc + st * (L::kTile / 16) + g * (kKeys * 8) + ks * 2, idesc(kKeys), hf + g + ks > 0 ? 1u : 0u);
          umma_commit(&s_full[h][st]);
          mbar_arrive(&s_full[h][st]);  // and orders the conversion's notes before the softmax
        }
        umma_commit(&k_empty[st]);
      }
      __syncwarp();
    };
    auto score = [&](unsigned no, int j) {
      if (j == 0 && !warp_wait(&q_full, items & 1, abort)) return false;
      if (!warp_wait(&k_full[no & 1], (no >> 1) & 1, abort)) return false;
      fence_after();
      if (no & 1) score_at(Const<1>{}); else score_at(Const<0>{});
      return true;
    };
    // (the same warp) O += P V
    auto product_at = [&](auto ST, int h, bool fresh) {
      constexpr int st = decltype(ST)::value;
      if (elected()) {
        const uint32_t base = tmem + h * 256;
#pragma unroll
        for (int hf = 0; hf < L::kHalves; ++hf)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)  // 32 keys' weights, hi and lo, lie in the 32 columns of their scores
            umma_tmem(base + 2 * kKeys, base + st * kKeys + (ks >> 1) * 32 + hf * 16 + (ks & 1) * 8, v_desc + st * (L::kTile / 16) + ks * 2,
                      idesc(D), hf + ks > 0 || !fresh ? 1u : 0u);
        umma_commit(&pv_done[h][st]);
        if (h == 1) umma_commit(&v_empty[st]);
      }
      __syncwarp();
    };
    auto product = [&](unsigned no, int j) {
      if (!warp_wait(&v_full[no & 1], (no >> 1) & 1, abort)) return false;
      const bool fresh = FP32 ? j % kFlush == 0 : j == 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a barrier a stage: a query tile may be done with the next key tile's weights before the other's are here)
        if (!warp_wait(&p_full[h][no & 1], (no >> 1) & 1, abort)) return false;
        fence_after();
        if (no & 1) product_at(Const<1>{}, h, fresh); else product_at(Const<0>{}, h, fresh);
      }
      return true;
    };
    for (int i = blockIdx.x; ok && i < work.total; i += gridDim.x) {
      const Item it = item_at(work, i);
      if (it.k0 >= it.k1) continue;
      const SeqInfo sq = info[it.s];
      const int32_t* table = a.b.tables + (size_t)it.s * a.g.max_pages;
      // the page numbers are asked for one tile before the rows, the rows one tile before they are converted
      auto page = [&](int row) { return row < sq.r ? table[row >> a.g.page_shift] : -1; };
      auto block = [&](int row, int pg) -> const uint8_t* {
        if (row >= sq.r) return nullptr;
        if ((unsigned)pg >= (unsigned)a.g.num_pages) {
          if (t == 0) flag(a.b.status, MBK_KV4_BAD_PAGE);
          return nullptr;
        }
        return a.g.pool + (size_t)pg * a.g.page_stride + (size_t)(a.layer * a.g.nkv + it.h) * a.g.head_stride +
               (unsigned)(((row & ((1 << a.g.page_shift) - 1)) / kRows) * a.g.block_bytes);
      };
      auto run = [&](auto& cur, auto& nxt, auto&& step) {
        {
          const int r = it.k0 * kKeys;
          cur.load(a, block(r, page(r)), block(r + kRows, page(r + kRows)), t);
        }
        int p0 = page((it.k0 + 1) * kKeys), p1 = page((it.k0 + 1) * kKeys + kRows);
        for (int k = it.k0; ok && k < it.k1; ++k, ++tile_no) {
          if (k + 1 < it.k1) {
            const int r = (k + 1) * kKeys;
            nxt.load(a, block(r, p0), block(r + kRows, p1), t);
            p0 = page(r + kKeys);
            p1 = page(r + kKeys + kRows);
          }
          ok = step(cur, k);
          cur = nxt;
        }
      };
      if (for_k) {
        RawK<D> cur, nxt;
        run(cur, nxt, [&](RawK<D>& w, int k) {
          const int st = tile_no & 1, slot = tile_no % kNotes;
          w.bad &= k * kKeys + kRows < sq.r ? 3u : 1u;  // a block behind the cache's end has no page: not an error
          if (tile_no >= 2 && !warp_wait(&k_empty[st], ((tile_no >> 1) - 1) & 1, abort)) return false;
          convert_k<D, FP32>(w, a, smem + L::kKAt + st * L::kTile, smem, slot, k * kKeys, sq.r, t, odd_group(k - it.k0), &notes[slot]);
          fence_async();
          mbar_arrive(&k_full[st]);
          return warp != 8 || (score(tile_no, k - it.k0) && (k == it.k0 || product(tile_no - 1, k - it.k0 - 1)));
        });
        if (ok && warp == 8) ok = product(tile_no - 1, it.k1 - it.k0 - 1);
      } else {
        RawV<D> cur, nxt;
        run(cur, nxt, [&](RawV<D>& w, int k) {
          const int st = tile_no & 1;
          if (tile_no >= 2 && !warp_wait(&v_empty[st], ((tile_no >> 1) - 1) & 1, abort)) return false;
          convert_v<D, FP32>(w, smem + L::kVAt + st * L::kTile, k * kKeys, sq.r, t, FP32 && odd_group(k - it.k0) ? ~0u : 0u);
          fence_async();
          mbar_arrive(&v_full[st]);
          return true;
        });
      }
      ++items;
    }
  } else {
    // ------------------------------------------------------------ softmax: one query row a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    const int h = warp >> 2, row = threadIdx.x & 127, lane = threadIdx.x & 31, wrow0 = (warp & 3) * 32;  // query tile, row, the warp's first
    const uint32_t mine = tmem + h * 256 + ((uint32_t)((warp & 3) * 32) << 16), t_out = mine + 2 * kKeys, t_sum = t_out + 64;  // this lane's columns
    bool ok = true;
    for (int i = blockIdx.x; ok && i < work.total; i += gridDim.x) {
      const Item it = item_at(work, i);
      const SeqInfo sq = info[it.s];
      if (it.k0 >= it.k1 && (it.parts > 0 || it.split > 0)) continue;
      const int qrow0 = it.tile * kItem + h * kQ, qrow = qrow0 + row, tok = qrow / a.by_grp, head = it.h * a.grp + qrow - tok * a.grp;
      const bool on = tok < sq.c;
      auto qpos_of = [&](int token) { return (FEAT && a.b.positions != nullptr ? a.b.positions[it.s] : sq.r - sq.c) + token; };
      const int limit = on ? sq.r - sq.c + tok : -1;
      const int first_limit = sq.r - sq.c + qrow0 / a.by_grp;
      const bool whole_tile = qrow0 + kQ <= sq.c * a.grp;
      // first row inside the window of this query and of the tile's last, where positions are the rows' numbers
      const bool by_row = FEAT && a.a.window > 0 && !a.g.track;
      const int low = by_row ? qpos_of(tok) - a.a.window + 1 : 0, last_low = by_row ? qpos_of(min(sq.c - 1, (qrow0 + kQ - 1) / a.by_grp)) - a.a.window + 1 : 0;
      const int qpos = FEAT && on ? qpos_of(tok) : 0;
      const float slope = FEAT && on && a.a.slopes != nullptr ? a.a.slopes[head] * kLog2e : 0.f;
      // The warp's 32 rows of q to the operand, each row's largest element scaled to [2^13, 2^14): neighbouring lanes read
      // a row's neighbouring 16 bytes (a row a thread would be 32 lines an instruction), all of them before the first is used.
      constexpr int kLanes = D * (FP32 ? 4 : 2) / 16, kRowsAtOnce = 32 / kLanes, kLoads = 32 / kRowsAtOnce;
      {
        uint4 q[kLoads];
        const unsigned char* base = reinterpret_cast<const unsigned char*>(a.a.q);
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          const int r = wrow0 + c * kRowsAtOnce + lane / kLanes, t = (qrow0 + r) / a.by_grp, hd = it.h * a.grp + qrow0 + r - t * a.grp;
          q[c] = make_uint4(0u, 0u, 0u, 0u);
          if (t < sq.c)
            q[c] = __ldg(reinterpret_cast<const uint4*>(base + ((size_t)(sq.tok0 + t) * a.a.ldq + (size_t)hd * D) * (FP32 ? 4 : 2)) + lane % kLanes);
        }
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
          float x[8], mx = 0.f, sum = 0.f;
          const uint32_t w[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
          if (FP32) {  // four dims; the neighbour has the other four of the eight
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float mine = __uint_as_float(w[e]), other = __shfl_xor_sync(0xffffffffu, mine, 1);
              x[e] = (lane & 1) ? other : mine;
              x[e + 4] = (lane & 1) ? mine : other;
              mx = fmaxf(mx, fabsf(mine));
              sum += mine;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[2 * e] = __uint_as_float(w[e] << 16);
              x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
              mx = fmaxf(mx, fmaxf(fabsf(x[2 * e]), fabsf(x[2 * e + 1])));
            }
          }
#pragma unroll
          for (int i = 1; i < kLanes; i <<= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
            if (FP32) sum += __shfl_xor_sync(0xffffffffu, sum, i);
          }
          int ex = (__float_as_int(mx) >> 23) & 255;
          ex = ex == 255 ? 140 : max(ex, 20);
          const float up = a.scale2 < 0.f ? -pow2i(140 - ex) : pow2i(140 - ex);  // mul >= 0: the largest acc is the largest score
          const int r = wrow0 + c * kRowsAtOnce + lane / kLanes;
          if (lane % kLanes == 0) row_scale[h * kQ + r] = make_float2(pow2i(ex - 140) * fabsf(a.scale2), sum * up);
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // the conversion's order of dims: 0 4 1 5 2 6 3 7
            const float x0 = x[e] * up, x1 = x[e + 4] * up;
            o[e] = pack_half(x0, x1);
            if (FP32 && (lane & 1)) {  // even lanes write hi, odd ones lo
              const float2 u = unpack_half(o[e]);
              o[e] = pack_half(x0 - u.x, x1 - u.y);
            }
          }
          const int chunk = FP32 ? (lane % kLanes) / 2 : lane % kLanes;
          unsigned char* to = smem + L::kQAt + h * L::kQTile + (chunk >> 3) * kQ * 128 + r * 128 + (((chunk & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(to + (FP32 && (lane & 1) ? kGroups * kQ * 128 : 0)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        __syncwarp();
      }
      const float mul = row_scale[h * kQ + row].x, addm = row_scale[h * kQ + row].y;  // score = mul * (acc, or fp32: scale_r acc + z_r addm)
      if (it.k0 < it.k1) {
        fence_async();
        mbar_arrive(&q_full);
      }
      float m = -INFINITY;
      f2 l = 0ull, z = 0ull;  // two partial sums each
      int e_cur = -15;
      unsigned nan_groups = 0u;
      for (int k = it.k0; k < it.k1; ++k, ++tile_no) {
        const int st = tile_no & 1, slot = tile_no % kNotes, j = k - it.k0;
        if (!(ok = warp_wait(&s_full[h][st], (tile_no >> 1) & 1, abort))) break;
        fence_after();
        f2 x[kKeys / 2];
        tmem_ld32(mine + st * kKeys, x);
        tmem_ld32(mine + st * kKeys + 32, x + 16);
        const float* pairs = reinterpret_cast<const float*>(smem + L::kPairsAt) + slot * 4 * kKeys;
        const TileNote note = notes[slot];
        tmem_wait_ld();
        if (FP32) {
          const f2 add = pair_of(addm, addm);
#pragma unroll
          for (int c = 0; c < kKeys / 2; c += 2) {
            const ulonglong2 sk = *reinterpret_cast<const ulonglong2*>(pairs + 2 * c), zk = *reinterpret_cast<const ulonglong2*>(pairs + kKeys + 2 * c);
            x[c] = fma2(sk.x, x[c], mul2(zk.x, add));
            x[c + 1] = fma2(sk.y, x[c + 1], mul2(zk.y, add));
          }
        }
        if (FEAT) {
          if (a.a.cap > 0.f) {  // cap tanh(x / cap) = cap - 2 cap / (1 + exp(2 x / cap))
            const f2 in = pair_of(mul * a.cap_in, mul * a.cap_in), one = pair_of(1.f, 1.f), out = pair_of(a.cap_out, a.cap_out),
                     out2 = pair_of(-2.f * a.cap_out, -2.f * a.cap_out);
#pragma unroll
            for (int c = 0; c < kKeys / 2; ++c) {
              float2 e = halves(mul2(x[c], in));
              e = halves(sum2(pair_of(ex2(e.x), ex2(e.y)), one));
              x[c] = fma2(pair_of(rcp(e.x), rcp(e.y)), out2, out);
            }
          } else {
            const f2 all = pair_of(mul, mul);
#pragma unroll
            for (int c = 0; c < kKeys / 2; ++c) x[c] = mul2(x[c], all);
          }
          // distances, where there is a bias or positions are not the rows' numbers
          if (a.a.slopes != nullptr || (a.a.window > 0 && a.g.track)) {
            const int* pos = reinterpret_cast<const int*>(smem + L::kPosAt) + slot * kKeys;
            const int win = a.a.window > 0 ? -a.a.window : -0x7fffffff - 1;
#pragma unroll
            for (int c = 0; c < kKeys / 2; ++c) {
              float2 v = halves(x[c]);
              const int at = k * kKeys + 2 * c;
              const int g0 = (a.g.track ? pos[2 * c] : at) - qpos, g1 = (a.g.track ? pos[2 * c + 1] : at + 1) - qpos;
              v.x = g0 <= win ? -INFINITY : fmaf(slope, (float)g0, v.x);
              v.y = g1 <= win ? -INFINITY : fmaf(slope, (float)g1, v.y);
              x[c] = pair_of(v.x, v.y);
            }
          }
        }
        if ((k + 1) * kKeys - 1 > first_limit || !whole_tile || note.bad != 0u || (FEAT && k * kKeys < last_low)) {
#pragma unroll
          for (int c = 0; c < kKeys / 2; ++c) {
            const int lim = (note.bad >> (c >> 4)) & 1u ? -1 : limit, at = k * kKeys + 2 * c;
            const float2 v = halves(x[c]);
            x[c] = pair_of(at > lim || (FEAT && at < low) ? -INFINITY : v.x, at + 1 > lim || (FEAT && at + 1 < low) ? -INFINITY : v.y);
          }
        }
        if ((note.nan[0][0] | note.nan[0][1] | note.nan[1][0] | note.nan[1][1]) != 0u) {
          // rows of V that are NaN: the output of those who see them is NaN
#pragma unroll
          for (int c = 0; c < kKeys / 2; ++c) {
            const float2 v = halves(x[c]);
            const unsigned b0 = note.nan[0][c >> 4] >> (2 * (c & 15)), b1 = note.nan[1][c >> 4] >> (2 * (c & 15));
            if (!(v.x == -INFINITY)) nan_groups |= (b0 & 1u) | (b1 & 1u) << 1;
            if (!(v.y == -INFINITY)) nan_groups |= (b0 >> 1 & 1u) | (b1 & 2u);
          }
        }
        float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < kKeys / 2; c += 2) {
          const float2 v = halves(x[c]), u = halves(x[c + 1]);
          top = fmaxf(top, fmaxf(v.x, v.y));
          top1 = fmaxf(top1, fmaxf(u.x, u.y));
        }
        top = fmaxf(top, top1);
        top = FEAT || top == -INFINITY ? top : top * mul;
        const int e_new = FP32 ? max(e_cur, max(note.e[0], note.e[1])) : 0;
        const bool renew = __any_sync(0xffffffffu, top > m + kSlack) || (FP32 && e_new != e_cur), flush = FP32 && j > 0 && j % kFlush == 0;
        float rescale = 1.f;
        if (renew) {
          const float nm = fmaxf(m, top);
          // (fp32: the weights' unit goes with V's largest scale; see below)
          rescale = nm == -INFINITY ? 1.f : ex2(m - nm + (FP32 ? (float)(e_cur - e_new) : 0.f));
          m = nm;
          l = mul2(l, pair_of(rescale, rescale));
          z = mul2(z, pair_of(rescale, rescale));
          e_cur = e_new;
        }
        if (j > 0 && (renew || flush)) {
          // the output, once the product before has left it
          if (!(ok = warp_wait(&pv_done[h][st ^ 1], ((tile_no - 1) >> 1) & 1, abort))) break;
          fence_after();
          if (flush) {  // moved to the sums
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
              const float sign = odd_group(j - 1) ? -1.f : 1.f;
              float o[16], s[16];
              tmem_ld16(t_out + c, o);
              if (j > kFlush) tmem_ld16(t_sum + c, s);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = (j > kFlush ? fmaf(sign, o[e], s[e]) : o[e]) * rescale;
              tmem_st16(t_sum + c, o);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < (FP32 && j > kFlush ? 128 : D); c += 16) {
              float o[16];
              tmem_ld16(t_out + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= rescale;
              tmem_st16(t_out + c, o);
            }
          }
        }
        // the weights, 32 keys at a time over their own scores: 16 columns of hi, fp32: 16 of lo
        // (fp32: times 2^(6 - e), e the exponent of V's largest scale: a weight of at most 2^8 times a scale is below 2^15)
        const float base = (m == -INFINITY ? 0.f : m) + (FP32 ? (float)(e_cur - 6) : 0.f);
        const f2 by = FEAT ? pair_of(1.f, 1.f) : pair_of(mul, mul), less = pair_of(-base, -base), minus = pair_of(-1.f, -1.f);
#pragma unroll
        for (int c0 = 0; c0 < kKeys / 2; c0 += 16) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float2 v = halves(fma2(x[c0 + c], by, less));
            f2 w = pair_of(ex2(v.x), ex2(v.y));
            l = sum2(l, w);
            if (FP32) {
              z = fma2(w, *reinterpret_cast<const f2*>(pairs + 3 * kKeys + 2 * (c0 + c)), z);
              w = mul2(w, *reinterpret_cast<const f2*>(pairs + 2 * kKeys + 2 * (c0 + c)));
            }
            v = halves(w);
            hi[c] = pack_half(v.x, v.y);
            if (FP32) {
              const float2 u = unpack_half(hi[c]);
              v = halves(fma2(pair_of(u.x, u.y), minus, w));
              lo[c] = pack_half(v.x, v.y);
            }
          }
          tmem_st16(mine + st * kKeys + 2 * c0, hi);
          if (FP32) tmem_st16(mine + st * kKeys + 2 * c0 + 16, lo);
        }
        tmem_wait_st();
        fence_before();
        mbar_arrive(&p_full[h][st]);
      }
      if (!ok) break;
      const int n = it.k1 - it.k0;
      if (n > 0) {
        if (!(ok = warp_wait(&pv_done[h][(tile_no - 1) & 1], ((tile_no - 1) >> 1) & 1, abort))) break;
        fence_after();
      }
      // the output, or the run's partial
      const bool last = it.parts <= 1;
      const float sign = FP32 && n > 0 && odd_group(n - 1) ? -1.f : 1.f;
      const float sum_l = halves(l).x + halves(l).y, sum_z = halves(z).x + halves(z).y;
      const float inv = last ? (sum_l > 0.f || sum_l != sum_l ? 1.f / sum_l : 0.f) : 1.f;
      const float m_ref = m + (FP32 ? (float)(e_cur - 6) : 0.f);  // what l and the output are relative to
      float* part = last ? nullptr : a.part + ((size_t)i * kItem + h * kQ) * (D + 4);
      // 32 columns of the warp's 32 rows at a time through shared memory (q's place: its products are done), so that a row's
      // bytes are written by neighbouring lanes
      unsigned char* stage = smem + L::kQAt + h * L::kQTile + wrow0 * 128;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        f2 o[16], s[16];
        __syncwarp();
        if (n > 0) {
          tmem_ld32(t_out + c0, o);
          if (FP32 && n > kFlush) tmem_ld32(t_sum + c0, s);
          tmem_wait_ld();
        }
        const bool bad = (nan_groups >> (c0 >> 6)) & 1u;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float4 v;
          float* y = &v.x;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f2 x = n > 0 ? o[2 * c + e] : 0ull;
            if (FP32 && n > kFlush) x = fma2(x, pair_of(sign, sign), s[2 * c + e]);
            if (FP32) x = sum2(x, pair_of(sum_z, sum_z));
            const float2 u = halves(mul2(x, pair_of(inv, inv)));
            y[2 * e] = bad ? NAN : n > 0 ? u.x : 0.f;
            y[2 * e + 1] = bad ? NAN : n > 0 ? u.y : 0.f;
          }
          *reinterpret_cast<float4*>(stage + lane * 128 + ((c ^ (lane & 7)) << 4)) = v;
        }
        __syncwarp();
#pragma unroll
        for (int r8 = 0; r8 < 8; ++r8) {
          const int r = r8 * 4 + (lane >> 3), c = lane & 7, t = (qrow0 + wrow0 + r) / a.by_grp, hd = it.h * a.grp + qrow0 + wrow0 + r - t * a.grp;
          const float4 v = *reinterpret_cast<const float4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
          if (t < sq.c) {
            const size_t at = (size_t)(sq.tok0 + t) * a.a.ldo + (size_t)hd * D + c0 + 4 * c;
            if (!last) {
              *reinterpret_cast<float4*>(part + (size_t)(wrow0 + r) * (D + 4) + c0 + 4 * c) = v;
            } else if (FP32) {
              *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.a.out) + at) = v;
            } else {
              const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y), q = __floats2bfloat162_rn(v.z, v.w);
              *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.a.out) + at) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
            }
          }
        }
      }
      if (on) {
        if (!last) {
          part[(size_t)row * (D + 4) + D] = m_ref;
          part[(size_t)row * (D + 4) + D + 1] = sum_l;
        } else if (a.lse != nullptr) {
          a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] = sum_l > 0.f ? m_ref + log2f(sum_l) : INFINITY;
        }
      }
      __syncwarp();
      fence_before();  // the output has been read before the next item's first product
    }
  }
  __syncwarp();
  __syncthreads();
  if (failed != 0u && threadIdx.x == 0) flag(a.b.status, MBK_KV4_TIMEOUT);
  if (failed != 0u && warp == 8) {
    // matrix instructions in flight end before their tensor memory is freed
    if (elected()) umma_commit(&drain);
    __syncwarp();
    for (int i = 0; i < 20000000 && !mbar_test(&drain, 0); ++i) {
    }
  }
  fence_before();
  __syncthreads();
  if (warp == 15) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Joins the runs of query tiles whose keys were split.
template <int D>
__global__ void __launch_bounds__(256) prompt_combine_kernel(const __grid_constant__ PromptArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int sums[16];
  const Work w = make_work(a, reinterpret_cast<SeqInfo*>(smem), sums, false);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kPiece = 32;  // rows at a time
  for (int x = blockIdx.x; x < w.total * (kItem / kPiece); x += gridDim.x) {
    const int i = x / (kItem / kPiece), row0 = x % (kItem / kPiece) * kPiece;
    const Item it = item_at(w, i);
    if (it.split != 0 || it.parts <= 1) continue;
    const SeqInfo sq = w.seq[it.s];
    const int rows = min(kPiece, sq.c * a.grp - it.tile * kItem - row0);
    if (rows <= 0) continue;
    // the splits of a (tile, head) are nkv items apart
    join<D>(a, sq, it.h, it.tile * kItem + row0, rows, it.parts, nullptr,
            [&](int k) { return a.part + ((size_t)(i + k * w.nkv) * kItem + row0) * (D + 4); });
  }
}

template <int D, bool FP32, bool FEAT>
cudaError_t run(const PromptArgs& a, cudaStream_t st) {
  static std::atomic<bool> once[64];
  const size_t smem = 1024 + Layout<D, FP32>::kInfoAt + (size_t)a.b.n_seq * sizeof(SeqInfo);
  if (cudaError_t e = allow_smem((const void*)prompt_kernel<D, FP32, FEAT>, once, 224 * 1024)) return e;
  const long long tiles = ((long long)a.b.max_count * a.grp + kItem - 1) / kItem;
  const long long items = a.b.n_seq * (long long)a.g.nkv * tiles * ((a.b.max_rows + kKeys - 1) / kKeys / kMinRun + 1);
  const int grid = (int)std::max<long long>(1, std::min<long long>(a.slots, items));
  if (cudaError_t e = launch(prompt_kernel<D, FP32, FEAT>, dim3(grid), kThreads, smem, st, false, a)) return e;
  return launch(prompt_combine_kernel<D>, dim3((unsigned)(4 * a.slots)), 256, (size_t)a.b.n_seq * sizeof(SeqInfo), st, true, a);
}

}  // namespace

size_t kv4_prompt_partials(const Kv4Geom& g, const Kv4Batch& b, int num_sms) {
  // split tiles are fewer than 2 x slots, and have at most kMaxRounds x slots runs and one more each
  const long long tiles = ((long long)b.max_count * (g.nq / g.nkv) + kItem - 1) / kItem * g.nkv * b.n_seq;
  const long long runs = (b.max_rows + kKeys - 1) / kKeys / kMinRun + 1;
  return (size_t)std::min<long long>((kMaxRounds + 2ll) * num_sms, tiles * runs) * kItem * (g.d + 4) * 4;
}

cudaError_t kv4_prompt(const Kv4Geom& g, int layer, const Kv4Batch& b, const Kv4Attn& at, int least, float* part, float* lse, int num_sms,
                       cudaStream_t st) {
  PromptArgs a;
  a.g = g;
  a.b = b;
  a.a = at;
  a.layer = layer;
  a.grp = g.nq / g.nkv;
  a.by_grp = ByGroup::of(a.grp);
  a.least = least;
  a.slots = num_sms;
  a.scale2 = at.scale * kLog2e;
  a.cap_in = at.cap > 0.f ? 2.f / at.cap : 0.f;
  a.cap_out = at.cap * kLog2e;
  a.part = part;
  a.lse = lse;
  // (a scale of zero times a masked score of -inf would be NaN: the general path scales first)
  const bool feat = at.cap > 0.f || at.slopes != nullptr || at.window > 0 || at.scale == 0.f;
  if (!at.bf16) return feat ? run<64, true, true>(a, st) : run<64, true, false>(a, st);
  if (g.d == 64) return feat ? run<64, false, true>(a, st) : run<64, false, false>(a, st);
  return feat ? run<128, false, true>(a, st) : run<128, false, false>(a, st);
}

}  // namespace mbk
