// mbk_kv4_attn.cu -- attention over a KV cache held in 4 bits, for a few query rows per KV head.
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
//   Bound by instructions, some 700 a block of 32 rows at head dim 128.  Measured: 64 ragged sequences of up to 16,384 rows,
// 32 query and 8 KV heads, d 128, bf16, capped: 664 MB in 142 us, 4.7 TB/s (69% of a copy's rate), issue slots 63% and the
// integer pipe 54% busy; one sequence of 130,001 rows, 9 and 3 heads, d 64, fp32: 28 MB in 19 us and 5 for the join, of which
// 4 would be the bytes': a warp has five blocks, and start, join and second launch are the rest.
#include "mbk_kv4_device.h"
#include "mbk_kv4_split.h"

namespace mbk {
namespace {

// MODE: what a tile's columns hold.
enum Mode {
  BF16_8 = 0,   // 8 bf16 queries
  BF16_16 = 1,  // 16 bf16 queries, two tiles
  FP32_4 = 2,   // 4 fp32 queries: hi | lo
  FP32_8 = 3,   // 8 fp32 queries, a tile of hi and one of lo
};
// FEAT: 0: one token per sequence, nothing but the scale; 1: with cap or bias; 2: anything.  Only the last
// has rows that some columns of a tile see and others do not, whose NaNs must be kept from the others.

// Warps of an attention CTA (one CTA per SM), within 227 KB of shared memory and 65,536 registers: 16 with
// 128 registers each, or 8 where the output takes too many of them.  Two blocks per warp are enough in the
// ring: at the memory's full rate a warp's turn comes every 1,600 (d 64) to 3,200 clocks, longer than a copy takes.
template <int D, int MODE>
struct Shape {
  static constexpr int kGroups = D / 64;
  static constexpr int NT = MODE == BF16_16 || MODE == FP32_8 ? 2 : 1;  // tiles of 8 columns
  static constexpr int NS = MODE == BF16_16 ? 2 : 1;                    // column sets with a softmax of their own
  static constexpr int TILE = MODE == BF16_16 ? 16 : MODE == FP32_4 ? 4 : 8;
  static constexpr bool kPrecise = MODE >= FP32_4;
  static constexpr int kWarps = D == 128 && NT == 2 ? 8 : 16;
  static constexpr int kStages = 2;
  static constexpr int kPart = D + 4;  // floats of a column's partial: o [d], m, l and 2 to keep 16-byte alignment
};

// ------------------------------------------------------------------ attention: the work and its split
// A segment is one (sequence, KV head, tile of query rows); its units are the blocks of 32 cache rows
// that it reads.  All segments' units, in order, are cut into equal runs, one per CTA and within it one
// per warp, whatever the sequences' lengths: a long context is spread over all SMs and a batch of
// short ones leaves none idle.  A segment inside one warp's run is written by the warp, one inside a
// CTA's run is joined in shared memory, the rest is joined by combine_kernel.
struct AttnArgs {
  Kv4Geom g;
  Kv4Batch b;
  Kv4Attn a;
  int layer, grp, grid_max, warps;
  ByGroup by_grp;
  int below;     // query rows per KV head from which on a sequence is the prompt kernel's, or 0
  float scale2, cap_in, cap_out;  // scale log2(e); 2 / cap, cap log2(e)
  float* part;   // [grid][2][tile columns][d + 4] partial (o, m, l) of segments that several CTAs share
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
  __device__ int tiles(const SeqInfo& q) const { return TILE == 0 ? 1 : (q.c * grp + TILE - 1) / max(TILE, 1); }  // 0: no tiles
  __device__ int units(const SeqInfo& q) const { return q.c == 0 ? 0 : tiles(q) * nkv * blocks(q); }
  // the run of CTA i: `base` units, one more for the first `extra` CTAs
  int base, extra;
  __device__ int begin(int i) const { return i * base + min(i, extra); }
  __device__ int cta_of(int u) const {
    const int big = extra * (base + 1);
    return u < big ? u / (base + 1) : extra + (u - big) / base;
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
  int carry = 0;
  if (a.b.n_seq <= 32) {
    // every warp for itself, without a barrier; all write the same
    const int s = threadIdx.x & 31;
    SeqInfo q{0, 0, 0, 0};
    int n = 0;
    if (s < a.b.n_seq) {
      const SeqView v = seq_view(a.g, a.b, s, report && threadIdx.x < 32);
      q.r = v.r;
      q.c = a.below == 0 || v.c * a.grp < a.below ? v.c : 0;  // longer ones are the prompt kernel's
      q.tok0 = v.tok0;
      n = sp.units(q);
    }
    int x = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, m);
      if (s >= m) x += y;
    }
    q.cum = x - n;
    if (s < a.b.n_seq) info[s] = q;
    carry = __shfl_sync(0xffffffffu, x, 31);
    __syncwarp();
  } else {
    for (int s0 = 0; s0 < a.b.n_seq; s0 += blockDim.x) {
      const int s = s0 + threadIdx.x;
      SeqInfo q{0, 0, 0, 0};
      int n = 0;
      if (s < a.b.n_seq) {
        const SeqView v = seq_view(a.g, a.b, s, report);
        q.r = v.r;
        q.c = a.below == 0 || v.c * a.grp < a.below ? v.c : 0;
        q.tok0 = v.tok0;
        n = sp.units(q);
      }
      int total;
      q.cum = carry + block_scan(n, warp_sums, &total);
      if (s < a.b.n_seq) info[s] = q;
      carry += total;
    }
    __syncthreads();
  }
  sp.total = carry;
  // one block for each warp of a CTA before a second CTA is used
  sp.grid = max(1, min(a.grid_max, (carry + a.warps - 1) / a.warps));
  sp.base = carry / sp.grid;
  sp.extra = carry - sp.base * sp.grid;
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

// ------------------------------------------------------------------ one block of 32 rows
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

// A lane's places in a stage: where its first 16-byte chunk of codes goes (the later ones differ from it in bits 5
// and 6 only), and where it reads K's rows 4 gid .., V's rows 8 tig .. and 8 tig + 4 ...
struct LaneAt {
  uint32_t put;
  int k, v0, v1;
};
template <int D>
__device__ __forceinline__ LaneAt lane_at(int lane) {
  constexpr int kGroups = D / 64;
  const int gid = lane >> 2, tig = lane & 3, r = lane / (2 * kGroups), in = lane % (2 * kGroups);
  return LaneAt{(uint32_t)((in >> 1) * 1024 + place(r) + (in & 1) * 16), place(4 * gid) + 8 * tig, place(8 * tig) + 4 * gid, place(8 * tig + 4) + 4 * gid};
}

// Copies a block to a stage: K (PARTS 1) or K and V (2), and the positions.
template <int D, int PARTS>
__device__ __forceinline__ void fetch(uint32_t st, const uint8_t* blk, bool pos, int lane, const LaneAt& at) {
  using S = Stage<D>;
  constexpr int kGroups = S::kGroups;
  const uint8_t* src = blk + lane * 16;
  const uint32_t put = st + at.put;  // stages begin at multiples of 128 bytes
#pragma unroll
  for (int sel = 0; sel < PARTS; ++sel)
#pragma unroll
    for (int i = 0; i < 2 * kGroups; ++i)  // chunk 32 i + lane: a row 16 / kGroups further each time
      cp16((put ^ (uint32_t)(i * (64 / kGroups))) + sel * S::kV, src + sel * half_bytes(D) + i * 512);
  // the pairs, 8 chunks a group, then the positions
  if (lane < PARTS * 8 * kGroups) {
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
  float mul[P::NS][2], add[P::kGroups][P::NS][2];  // score = mul * sum of (scale_r * acc + z_r * add), in the base-2 logarithm's units
  float mid[P::kGroups][2];                        // fp32: -7.5 add: codes count from their middle
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
    const int row = tile * P::TILE + col, tok = row / a.by_grp, head = h * a.grp + row - tok * a.grp;
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
      t.mul[ns][j] = __shfl_sync(0xffffffffu, down, from) * a.scale2;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const float sg = __shfl_sync(0xffffffffu, sum[g], from);
        t.add[g][ns][j] = sg * (1.f / 16777216.f) * __shfl_sync(0xffffffffu, up, from);  // sum(q) in acc's units
        if (P::kPrecise) {
          t.mid[g][j] = MODE == FP32_4 && tig >= 2 ? 0.f : -7.5f * t.add[g][ns][j];  // the lo columns start at zero
        }
      }
      const int crow = tile * P::TILE + column<MODE>(tig, ns, j), ctok = crow / a.by_grp;
      const bool con = ctok < sq.c;
      t.limit[ns][j] = con ? sq.r - sq.c + ctok : -1;
      if (FEAT > 0) {
        t.qpos[ns][j] = con ? (a.b.positions != nullptr ? a.b.positions[s] : sq.r - sq.c) + ctok : 0;
        t.slope[ns][j] = con && a.a.slopes != nullptr ? a.a.slopes[h * a.grp + crow - ctok * a.grp] * kLog2e : 0.f;
      }
    }
  }
}

// Scores of the tile against a staged block, in units of the base-2 logarithm: sc[ns][i][j] is cache row
// 32 blk + 4 gid + i against the lane's column j of set ns; -inf where the row is not visible.
// full: every row of the block is visible to every query of the tile (a window aside).
template <int D, int MODE, int FEAT>
__device__ __forceinline__ void scores(const QTile<D, MODE>& t, const AttnArgs& a, const unsigned char* st, int blk, bool full, int lane,
                                       const LaneAt& at, float (&sc)[Shape<D, MODE>::NS][4][2]) {
  using S = Stage<D>;
  using P = Shape<D, MODE>;
  constexpr int kGroups = P::kGroups, NS = P::NS, NT = P::NT;
  const int gid = lane >> 2;
  // row 4 gid + i lies at place(4 gid) + 128 i
  const unsigned char* kb = st + at.k;
  uint32_t pr[kGroups * 4];
#pragma unroll
  for (int i = 0; i < kGroups; ++i)
    *reinterpret_cast<uint4*>(pr + 4 * i) = *reinterpret_cast<const uint4*>(st + S::kCodes + gid * (16 * kGroups) + 16 * i);
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {  // tile rows gid: cache row 4 gid + 2 mt; gid + 8: the next one
      const uint2 w0 = *reinterpret_cast<const uint2*>(kb + g * 1024 + 256 * mt);
      const uint2 w1 = *reinterpret_cast<const uint2*>(kb + g * 1024 + 256 * mt + 128);
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
            float& x = sc[ns][2 * mt + i][j];
            x = fmaf(p.x, acc, g == 0 ? z * t.add[g][ns][j] : fmaf(z, t.add[g][ns][j], x));
          }
      }
    }
  }
  const int r0 = blk * kRows + 4 * gid;
  // one branch per feature, not per score: the eight scores then go through it side by side
  if (FEAT > 0 && a.a.cap > 0.f) {
#pragma unroll
    for (int i = 0; i < 4 * NS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // cap tanh(x / cap) = cap (1 - 2 / (1 + exp(2 x / cap))): off by a few 2^-24 of cap
        float& x = sc[i / 4][i % 4][j];
        x = fmaf(-2.f * a.cap_out, rcp(1.f + ex2(x * (t.mul[i / 4][j] * a.cap_in))), a.cap_out);
      }
  } else {
#pragma unroll
    for (int i = 0; i < 4 * NS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) sc[i / 4][i % 4][j] *= t.mul[i / 4][j];
  }
  if (FEAT > 0 && (a.a.slopes != nullptr || (FEAT == 2 && a.a.window > 0))) {
    int kpos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) kpos[i] = r0 + i;
    if (a.g.track) *reinterpret_cast<int4*>(kpos) = *reinterpret_cast<const int4*>(st + S::kPos + 16 * gid);
#pragma unroll
    for (int i = 0; i < 4 * NS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float& x = sc[i / 4][i % 4][j];
        const int gap = kpos[i % 4] - t.qpos[i / 4][j];
        x = fmaf(t.slope[i / 4][j], (float)gap, x);  // without slopes: 0, which leaves x as it is
        if (FEAT == 2) x = a.a.window > 0 && gap <= -a.a.window ? -INFINITY : x;
      }
  }
  if (!full) {
#pragma unroll
    for (int i = 0; i < 4 * NS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) sc[i / 4][i % 4][j] = r0 + i % 4 <= t.limit[i / 4][j] ? sc[i / 4][i % 4][j] : -INFINITY;
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
__device__ __forceinline__ void accumulate(Acc<D, MODE>& A, const unsigned char* st, int blk, int rows, int lane, const LaneAt& at,
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
  // how far the scores exceed their columns' reference (a reference of -inf: by -inf or inf; NaN does not count)
  float over = -INFINITY;
#pragma unroll
  for (int ns = 0; ns < NS; ++ns)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      over = fmaxf(over, fmaxf(fmaxf(sc[ns][0][j], sc[ns][1][j]), fmaxf(sc[ns][2][j], sc[ns][3][j])) - fmaxf(A.m[ns][j], -3e38f));
  if (__any_sync(0xffffffffu, (over > kSlack) | (eb > A.e))) {
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
  const unsigned char *v0 = st + S::kV + at.v0, *v1 = st + S::kV + at.v1;
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
    // codes count from their middle: sum p (code - 7.5) is of the output's size, sum p code many times that.  Truncation
    // leaves a bias in each block's share all the same, which grew against the output as its rows' average shrinks (9e-6 at
    // 130,001 rows); so every other block takes 15 - code and is subtracted, and the biases cancel.
    const float sign = P::kPrecise && (blk & 1) ? -1.f : 1.f;
    const uint32_t flip = P::kPrecise && (blk & 1) ? ~0u : 0u;
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
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // row 8 tig + i lies at place(8 tig) + 128 i, row 8 tig + 4 + i at place(8 tig + 4) + 128 i
      w[i] = *reinterpret_cast<const uint32_t*>(v0 + g * 1024 + 128 * i);
      w[i + 4] = *reinterpret_cast<const uint32_t*>(v1 + g * 1024 + 128 * i);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // codes 4 half .. + 3 of the word: dims 8 gid + 4 half ..
      const uint32_t sel = half ? 0x7632u : 0x5410u;
      uint32_t x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) codes<P::kPrecise>(__byte_perm(w[i], w[i + 4], sel), x[i], flip);
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
          if (P::kPrecise) {
            add2(o[0], o[1], c[0], c[1], sign);
            add2(o[2], o[3], c[2], c[3], sign);
          } else {
            add2(o[0], o[1], c[0], c[1]);
            add2(o[2], o[3], c[2], c[3]);
          }
        }
    }
  }
}

__device__ __forceinline__ float all_rows(float x) {  // sum over the lanes of a column
#pragma unroll
  for (int m = 4; m < 32; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// The end of a tile's run: the sums over the columns' lanes; then either the output itself or the
// partial (o [d], m, l) of each column at `dep`, kPart floats apart.
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
      const int col = column<MODE>(tig, ns, j), row = tile * P::TILE + col, tok = row / a.by_grp, head = h * a.grp + row - tok * a.grp;
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
          store8(dep + col * P::kPart + 64 * g + 8 * gid, x);
        } else {
          store_out(a.a, (size_t)(sq.tok0 + tok) * a.a.ldo + (size_t)head * D + 64 * g + 8 * gid, x);
        }
      }
      if (on && gid == 0) {
        if (dep != nullptr) {
          dep[col * P::kPart + D] = A.m[ns][j];
          dep[col * P::kPart + D + 1] = l;
        } else if (a.lse != nullptr) {
          a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] = l > 0.f ? A.m[ns][j] + log2f(l) : INFINITY;
        }
      }
    }
}

template <int D, int MODE, int FEAT>
__global__ void __launch_bounds__(Shape<D, MODE>::kWarps * 32) attn_kernel(const __grid_constant__ AttnArgs a) {
  using P = Shape<D, MODE>;
  using S = Stage<D>;
  constexpr int TILE = P::TILE, kWarps = P::kWarps, kStages = P::kStages;
  static_assert(kStages * S::kBytes >= TILE * P::kPart * 4, "a warp's last partial lies in its ring");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int warp_sums[kWarps];
  __shared__ int dep_seg[kWarps][2];  // first unit of the segment of a warp's partial, or -1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  SeqInfo* info = reinterpret_cast<SeqInfo*>(smem);
  unsigned char* ring = smem + ((size_t)a.b.n_seq * sizeof(SeqInfo) + 127) / 128 * 128;
  // a warp's first partial (its run goes on) beside the rings, its last one in its own ring
  float* deps = reinterpret_cast<float*>(ring + (size_t)kWarps * kStages * S::kBytes);
  const int dep_floats = min(TILE, a.b.max_count * a.grp) * P::kPart;
  auto dep_at = [&](int k) {  // k = 2 warp + slot
    return (k & 1) ? reinterpret_cast<float*>(ring + (size_t)(k >> 1) * kStages * S::kBytes) : deps + (size_t)(k >> 1) * dep_floats;
  };
  const Split<TILE> sp = make_split<TILE>(a, info, warp_sums, blockIdx.x == 0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane < 2) dep_seg[warp][lane] = -1;
  __syncthreads();
  if ((int)blockIdx.x >= sp.grid || sp.total == 0) return;
  const int c0 = sp.begin(blockIdx.x), c1 = sp.begin(blockIdx.x + 1), cn = c1 - c0;
  const int wb = cn / kWarps, we = cn % kWarps;
  const int u0 = c0 + warp * wb + min(warp, we), u1 = u0 + wb + (warp < we ? 1 : 0);
  unsigned char* mine = ring + (size_t)warp * kStages * S::kBytes;
  const uint32_t mine_s = smem_of(mine);

  if (u0 < u1) {
    const bool need_pos = FEAT > 0 && a.g.track;
    Seg ps = locate(sp, u0);  // the copies' segment
    Seg cs = ps;              // the arithmetic's
    SeqInfo psq = info[ps.s], csq = psq;
    unsigned have = 0;        // bit i: stage i holds a block to be used
    auto last_row = [&](const Seg& g, const SeqInfo& q) {  // last row that any query of the tile sees
      const int tok = min(q.c - 1, (g.tile * TILE + TILE - 1) / a.by_grp);
      return q.r - q.c + tok;
    };
    int plast = last_row(ps, psq);
    const int32_t* table = a.b.tables + (size_t)ps.s * a.g.max_pages;
    const int page_mask = (1 << a.g.page_shift) / kRows - 1;
    auto page_of = [&](int blk) { return blk * kRows <= plast ? table[blk * kRows >> a.g.page_shift] : 0; };
    {  // the first queries are asked for before the page numbers are waited for
      const int row = cs.tile * TILE + (lane >> 2) % TILE, tok = row / a.by_grp;
      if (tok < csq.c) {
        const size_t from = (size_t)(csq.tok0 + tok) * a.a.ldq + (size_t)(cs.h * a.grp + row - tok * a.grp) * D;
        constexpr int kBytes = P::kPrecise ? 4 : 2;
        const unsigned char* p = reinterpret_cast<const unsigned char*>(a.a.q) + from * kBytes + (lane & 3) * (D * kBytes / 4);
        asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
      }
    }
    int page = page_of(ps.first + u0 - ps.u0);  // of the next block to be copied, asked for one block ahead
    const LaneAt at = lane_at<D>(lane);
    const uint8_t* src = nullptr;  // the block copied last
    bool fresh = true;
    auto issue = [&](int u) {
      if (u < u1) {
        if (u >= ps.u0 + ps.n) {
          ps = locate(sp, u);
          psq = info[ps.s];
          plast = last_row(ps, psq);
          table = a.b.tables + (size_t)ps.s * a.g.max_pages;
          page = page_of(ps.first);
          fresh = true;
        }
        const int blk = ps.first + u - ps.u0, stg = (u - u0) % kStages;
        have &= ~(1u << stg);
        if (blk * kRows <= plast) {
          if (fresh) {  // the first block of a page, or of the run
            src = nullptr;
            if ((unsigned)page < (unsigned)a.g.num_pages)
              src = a.g.pool + (size_t)page * a.g.page_stride + (size_t)(a.layer * a.g.nkv + ps.h) * a.g.head_stride +
                    (unsigned)((blk & page_mask) * a.g.block_bytes);
            else if (lane == 0)
              flag(a.b.status, MBK_KV4_BAD_PAGE);
          } else if (src != nullptr) {
            src += a.g.block_bytes;
          }
          if (src != nullptr) {
            have |= 1u << stg;
            fetch<D, 2>(mine_s + stg * S::kBytes, src, need_pos, lane, at);
          }
          fresh = ((blk + 1) & page_mask) == 0;
          if (fresh) page = page_of(blk + 1);
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
      const int first_limit = csq.r - csq.c + (cs.tile * TILE) / a.by_grp;
      const int end = min(u1, cs.u0 + cs.n);
      for (; u < end; ++u) {
        const int stg = (u - u0) % kStages, blk = cs.first + u - cs.u0;
        const bool use = (have >> stg) & 1u;
        issue(u + kStages - 1);  // into the stage that the iteration before has read
        cp_wait<kStages - 1>();
        __syncwarp();
        if (use) {
          const unsigned char* st = mine + stg * S::kBytes;
          float sc[P::NS][4][2];
          scores<D, MODE, FEAT>(qt, a, st, blk, (blk + 1) * kRows - 1 <= first_limit, lane, at, sc);
          accumulate<D, MODE, FEAT>(acc, st, blk, csq.r, lane, at, sc);
        }
        __syncwarp();
      }
      float* dep = nullptr;
      if (cs.u0 < u0 || cs.u0 + cs.n > u1) {
        const int slot = cs.u0 < u0 ? 0 : 1;  // it began in an earlier warp's run, or goes on in a later one's
        if (lane == 0) dep_seg[warp][slot] = cs.u0;
        dep = dep_at(2 * warp + slot);
      }
      finish<D, MODE>(acc, a, csq, cs.h, cs.tile, lane, dep);
    }
  }
  __syncthreads();
  // Join the warps' partials, a warp for each column of each segment.  They lie in the order of the warps, and those of a
  // segment are its first warp's last one (slot 1, unless it began before this CTA) and then first ones (slot 0).
  // Lane e looks at entry e = 2 warp + slot.
  int seg = -1, ahead0 = -1, ahead1 = -1;
  if (lane < 2 * kWarps) {
    seg = dep_seg[lane >> 1][lane & 1];
    if (lane >= 2) {
      ahead0 = dep_seg[(lane >> 1) - 1][0];
      ahead1 = dep_seg[(lane >> 1) - 1][1];
    }
  }
  unsigned starts = __ballot_sync(0xffffffffu, seg >= 0 && ((lane & 1) || (seg != ahead0 && seg != ahead1)));
  const int cols_max = dep_floats / P::kPart;
  int turn = 0;
  for (; starts != 0u; starts &= starts - 1) {
    const int e = __ffs(starts) - 1, mine_seg = __shfl_sync(0xffffffffu, seg, e);
    const unsigned more = __ballot_sync(0xffffffffu, seg == mine_seg && !(lane & 1) && lane > e);
    const int n = 1 + __popc(more);
    int col = (warp - turn) & (kWarps - 1);  // this warp's column of the segment, if it has one
    turn += cols_max;
    if (col >= cols_max) continue;
    const Seg g = locate(sp, mine_seg);
    const SeqInfo sq = info[g.s];
    float* to = g.u0 >= c0 && g.u0 + g.n <= c1 ? nullptr : a.part + ((size_t)blockIdx.x * 2 + (g.u0 < c0 ? 0 : 1)) * TILE * P::kPart;
    for (; col < min(TILE, sq.c * a.grp - g.tile * TILE); col += kWarps)
      join_column<D>(a, sq, g.h, g.tile * TILE, col, n, to, [&](int k) { return k == 0 ? dep_at(e) : dep_at(2 * ((e >> 1) + k)); });
  }
}

// Joins the partials of segments that several CTAs share; grid: (KV heads x tiles at most, sequences).
template <int D, int TILE>
__global__ void __launch_bounds__(512) combine_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int warp_sums[16];
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
    join<D>(a, sq, h, tile * TILE, min(TILE, sq.c * a.grp - tile * TILE), last - first + 1, nullptr,
            [&](int k) { return a.part + ((size_t)(first + k) * 2 + (k == 0 ? 1 : 0)) * TILE * (D + 4); });
  }
}

// The weight that each cache row got: weight_r += sum over the sequence's queries and the group's heads
// of exp2(score - lse).  A warp owns a block's 32 rows and goes through all the query tiles, so the
// sums have one order and no atomics; the scores are computed again from K (half a row's bytes)
// rather than kept, which would cost 4 bytes written and read for each of the group's heads.  Bound by instructions, as
// attn_kernel: 48 ragged sequences of up to 8,191 rows, 14 and 2 heads, d 64: 15.5 us (attention 23, join 6.4).
constexpr int kWeightWarps = 8;
template <int D, int MODE, int FEAT>
__global__ void __launch_bounds__(kWeightWarps * 32) weight_kernel(const __grid_constant__ AttnArgs a) {
  using P = Shape<D, MODE>;
  using S = Stage<D>;
  constexpr int TILE = P::TILE;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int warp_sums[kWeightWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  SeqInfo* info = reinterpret_cast<SeqInfo*>(smem);
  unsigned char* mine = smem + ((size_t)a.b.n_seq * sizeof(SeqInfo) + 127) / 128 * 128 + (size_t)warp * 2 * S::kBytes;
  const Split<0> sp = make_split<0>(a, info, warp_sums, false);
  if ((int)blockIdx.x >= sp.grid || sp.total == 0) return;
  const int c0 = sp.begin(blockIdx.x), cn = sp.begin(blockIdx.x + 1) - c0, wb = cn / kWeightWarps, we = cn % kWeightWarps;
  const int u0 = c0 + warp * wb + min(warp, we), u1 = u0 + wb + (warp < we ? 1 : 0);
  if (u0 >= u1) return;
  Seg ps = locate(sp, u0);
  const LaneAt here = lane_at<D>(lane);
  uint8_t* next = nullptr;  // the block that is being copied
  auto issue = [&](int u) {
    next = nullptr;
    if (u < u1) {
      if (u >= ps.u0 + ps.n) ps = locate(sp, u);
      const int blk = ps.first + u - ps.u0;
      if (blk * kRows < info[ps.s].r) next = block_of(a.g, a.b.tables + (size_t)ps.s * a.g.max_pages, a.layer, ps.h, blk * kRows, nullptr);
      if (next != nullptr) fetch<D, 1>(smem_of(mine) + ((u - u0) & 1) * S::kBytes, next, FEAT > 0, lane, here);
    }
    cp_commit();
  };
  issue(u0);
  Seg cs = ps;
  QTile<D, MODE> qt;
  float lse[P::NS][2];
  bool fresh = true;  // the queries of cs are not loaded yet
  for (int u = u0; u < u1; ++u) {
    uint8_t* p = next;
    issue(u + 1);
    if (u >= cs.u0 + cs.n) {
      cs = locate(sp, u);
      fresh = true;
    }
    const SeqInfo sq = info[cs.s];
    const int blk = cs.first + u - cs.u0, tiles = (sq.c * a.grp + TILE - 1) / TILE;
    float* at = reinterpret_cast<float*>(p + weight_at(D)) + 4 * gid;
    float w[4] = {0.f, 0.f, 0.f, 0.f}, old[4];
    if (p != nullptr && tig == 0) *reinterpret_cast<float4*>(old) = *reinterpret_cast<const float4*>(at);
    const unsigned char* st = mine + ((u - u0) & 1) * S::kBytes;
    for (int tile = 0; tile < tiles; ++tile) {
      const int last = sq.r - sq.c + min(sq.c - 1, (tile * TILE + TILE - 1) / a.by_grp), first = sq.r - sq.c + (tile * TILE) / a.by_grp;
      if (p == nullptr || blk * kRows > last) continue;
      if (fresh || tiles > 1) {
        load_q<D, MODE, FEAT>(qt, a, sq, cs.s, cs.h, tile, lane);
#pragma unroll
        for (int ns = 0; ns < P::NS; ++ns)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int row = tile * TILE + column<MODE>(tig, ns, j), tok = row / a.by_grp, head = cs.h * a.grp + row - tok * a.grp;
            // columns that hold no query, and the lo halves, add nothing
            lse[ns][j] = tok < sq.c && !(MODE == FP32_4 && tig >= 2) ? a.lse[(size_t)(sq.tok0 + tok) * a.g.nq + head] : INFINITY;
          }
        fresh = false;
      }
      cp_wait<1>();
      __syncwarp();
      float sc[P::NS][4][2];
      scores<D, MODE, FEAT>(qt, a, st, blk, (blk + 1) * kRows - 1 <= first, lane, here, sc);
#pragma unroll
      for (int ns = 0; ns < P::NS; ++ns)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] += lse[ns][j] == INFINITY ? 0.f : ex2(sc[ns][i][j] - lse[ns][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
    }
    if (p != nullptr && tig == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (blk * kRows + 4 * gid + i < sq.r) at[i] = old[i] + w[i];
    }
    __syncwarp();
  }
}

constexpr int kAttnSmem = 226 * 1024;  // dynamic shared memory at most: 227 KB less the static part

// Units of the batch at most.
long long max_units(const Kv4Geom& g, const Kv4Batch& b, int tile) {
  const long long tiles = ((long long)b.max_count * (g.nq / g.nkv) + tile - 1) / tile;
  return (long long)b.n_seq * g.nkv * tiles * std::max(1, (b.max_rows + kRows - 1) / kRows);
}

template <int D, int MODE, int FEAT>
cudaError_t run_attention(AttnArgs a, bool others, int num_sms, cudaStream_t st) {
  constexpr int TILE = Shape<D, MODE>::TILE, kWarps = Shape<D, MODE>::kWarps, kStages = Shape<D, MODE>::kStages;
  a.warps = kWarps;
  using S = Stage<D>;
  static std::atomic<bool> once[64], once_w[64];
  const size_t info = ((size_t)a.b.n_seq * sizeof(SeqInfo) + 127) / 128 * 128;
  const int dep_rows = std::min<long long>(TILE, (long long)a.b.max_count * a.grp);
  const size_t smem = info + (size_t)kWarps * kStages * S::kBytes + (size_t)kWarps * dep_rows * Shape<D, MODE>::kPart * 4;
  if (cudaError_t e = allow_smem((const void*)attn_kernel<D, MODE, FEAT>, once, kAttnSmem)) return e;
  const long long units = max_units(a.g, a.b, TILE);
  const int grid = (int)std::max<long long>(1, std::min<long long>(num_sms, (units + kWarps - 1) / kWarps));
  if (others)
    if (cudaError_t e = launch(attn_kernel<D, MODE, FEAT>, dim3(grid), kWarps * 32, smem, st, false, a)) return e;
  if (others && grid > 1) {
    const long long segs = (long long)a.g.nkv * (((long long)a.b.max_count * a.grp + TILE - 1) / TILE);
    if (cudaError_t e = launch(combine_kernel<D, TILE>, dim3((unsigned)std::min<long long>(segs, 4096), a.b.n_seq), 512, info, st, true, a)) return e;
  }
  if (a.lse != nullptr) {
    if (cudaError_t e = allow_smem((const void*)weight_kernel<D, MODE, FEAT>, once_w, kAttnSmem)) return e;
    a.warps = kWeightWarps;
    a.below = 0;  // every sequence's rows
    a.grid_max = 2 * num_sms;
    const long long blocks = (long long)a.b.n_seq * a.g.nkv * std::max(1, (a.b.max_rows + kRows - 1) / kRows);
    const int wg = (int)std::max<long long>(1, std::min<long long>(a.grid_max, (blocks + kWeightWarps - 1) / kWeightWarps));
    return launch(weight_kernel<D, MODE, FEAT>, dim3(wg), kWeightWarps * 32, info + (size_t)kWeightWarps * 2 * S::kBytes, st, false, a);
  }
  return cudaSuccess;
}

template <int D, int MODE>
cudaError_t pick_feat(const AttnArgs& a, bool others, int num_sms, cudaStream_t st) {
  if (a.b.max_count > 1 || a.a.window > 0) return run_attention<D, MODE, 2>(a, others, num_sms, st);
  if (a.a.cap > 0.f || a.a.slopes != nullptr) return run_attention<D, MODE, 1>(a, others, num_sms, st);
  return run_attention<D, MODE, 0>(a, others, num_sms, st);
}

// The narrowest tile that holds a sequence's queries of one KV head, or else the widest.
template <int D>
cudaError_t pick_attention(const AttnArgs& a, bool others, int num_sms, cudaStream_t st) {
  const long long cols = (long long)a.b.max_count * a.grp;
  if (a.a.bf16) return cols <= 8 ? pick_feat<D, BF16_8>(a, others, num_sms, st) : pick_feat<D, BF16_16>(a, others, num_sms, st);
  return cols <= 4 ? pick_feat<D, FP32_4>(a, others, num_sms, st) : pick_feat<D, FP32_8>(a, others, num_sms, st);
}

// Query rows per KV head from which on a sequence goes to the prompt kernel.  That one takes 256 query rows at a time
// and 26 to 38 us however few keys there are; the decode kernel's time grows with rows x keys, 8 or 16 query rows at a
// time.  Measured (us, decode / prompt; with N the (sequence, KV head) pairs and R the rows):
//   fp32 d 64, N 3:    R 512 at 510 rows 14 / 38;   R 4096 at 255 21 / 40, at 510 32 / 40;  R 32768 at 159 58 / 66, at 255 85 / 67
//   fp32 d 64, N 48:   R 512 at 192 37 / 46, at 318 52 / 51;   R 2048 at 126 56 / 63, at 192 78 / 61
//   bf16 d 64, N 128:  R 512 at 96 34 / 37, at 160 47 / 38;    R 2048 at 160 94 / 107, at 256 140 / 111
//   bf16 d 128, N 8:   R 512 at 512 26 / 34;   R 4096 at 192 35 / 40, at 320 46 / 48;       R 32768 at 128 108 / 109
//   bf16 d 128, N 128: R 512 at 64 40 / 46, at 128 61 / 47
// so the border is near 100 query rows where there is much to do and moves up as 1 / (N R).
long long prompt_rows(const Kv4Geom& g, const Kv4Batch& b) {
  return 96 + (1ll << 22) / ((long long)b.n_seq * g.nkv * std::max(1, b.max_rows));
}

// Whether the batch may have a sequence for the prompt kernel (fp32 at head dim 128 would need two accumulators and
// operands twice as large per tile: the decode kernel takes it).
bool has_prompts(const Kv4Geom& g, const Kv4Batch& b, int bf16) {
  return (long long)b.max_count * (g.nq / g.nkv) >= prompt_rows(g, b) && (bf16 || g.d == 64);
}
// The workspace: the decode kernel's partials, the prompt kernel's, lse.
size_t own_bytes(const Kv4Geom& g, const Kv4Batch& b, int num_sms) {
  // none where one CTA's warps have a block each, whatever the queries' type (tiles of 4 at least)
  return max_units(g, b, 4) <= (g.d == 64 ? 16 : 8) ? 0 : round256((size_t)num_sms * 2 * 16 * (g.d + 4) * 4);
}
size_t part_bytes(const Kv4Geom& g, const Kv4Batch& b, int num_sms) {
  return own_bytes(g, b, num_sms) +
         ((long long)b.max_count * (g.nq / g.nkv) >= prompt_rows(g, b) ? round256(kv4_prompt_partials(g, b, num_sms)) : 0);
}

}  // namespace

size_t kv4_attention_workspace(const Kv4Geom& g, const Kv4Batch& b, int num_sms) {
  return part_bytes(g, b, num_sms) + (g.track ? round256((size_t)b.n_tokens * g.nq * 4) : 0);
}

cudaError_t kv4_attention(const Kv4Geom& g, int layer, const Kv4Batch& b, Kv4Attn at, void* ws, int num_sms, cudaStream_t st) {
  if (!g.track) at.window = std::min(at.window, 1 << 28);  // row numbers are below 2^27: no more than all, and sums stay in 32 bits
  AttnArgs a;
  a.g = g;
  a.b = b;
  a.a = at;
  a.layer = layer;
  a.grp = g.nq / g.nkv;
  a.by_grp = ByGroup::of(a.grp);
  a.grid_max = num_sms;
  a.scale2 = at.scale * kLog2e;
  a.cap_in = at.cap > 0.f ? 2.f / at.cap : 0.f;
  a.cap_out = at.cap * kLog2e;
  a.part = reinterpret_cast<float*>(ws);
  a.lse = at.accumulate ? reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + part_bytes(g, b, num_sms)) : nullptr;
  a.below = 0;
  const bool prompts = has_prompts(g, b, at.bf16);
  if (prompts) {
    // a sequence alone goes to the prompt kernel however few its tokens turn out to be
    a.below = b.n_seq == 1 ? 1 : (int)prompt_rows(g, b);
    uint8_t* part = reinterpret_cast<uint8_t*>(ws) + own_bytes(g, b, num_sms);
    if (cudaError_t e = kv4_prompt(g, layer, b, at, a.below, reinterpret_cast<float*>(part), a.lse, num_sms, st)) return e;
  }
  const bool others = !prompts || b.n_seq > 1;
  return g.d == 64 ? pick_attention<64>(a, others, num_sms, st) : pick_attention<128>(a, others, num_sms, st);
}

}  // namespace mbk
