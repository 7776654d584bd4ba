// Attention of a few query rows over the pages of the 8-bit cache.
//
// For every query row i of a kv head's group:  o_i = sum_j p_ij s_v(j) c_v,j / sum_j p_ij,
// p_ij = exp(s_ij - m_i), s_ij the modified scores of (q_i . c_k,j) s_k(j), with codes c
// and the scale s of the page that j lies on.
//
// Bound: memory (2 d bytes a token and kv head, read once for each block of query rows:
// of 8 rows, or of up to 32 where the page tables have room for more than L2 holds).  The keys
// of all (sequence, kv head, block of query rows) are cut into tiles of 32 tokens
// and numbered; every warp of the grid takes an equal, contiguous run of tiles, so
// ragged lengths, few long sequences and many short ones all fill the SMs alike.
// A warp works alone: one thread of it brings tiles in by TMA (128-byte swizzle, a ring of
// units, tiles of keys and of values in turn, the scales by 4-byte copies on the same barrier),
// and the warp multiplies with mma.sync m16n8k16, f16 operands, fp32 sums:
//     S^T = K Q^T   (A: 16 tokens x 16 dims of codes; B: 8 query rows)
//     O^T = V^T P^T (A: 16 dims x 16 tokens of codes; B: weights)
// Few rows fill an 8-wide B operand, not the 128 rows of a tcgen05 tile, and the
// codes become f16 in registers on their way into A (an int8 or e4m3 code is exact
// in f16, so no scale enters before the fp32 sums); a tcgen05 operand would have to
// go back to shared memory at twice the bytes.  The dims of Q are permuted so that a
// thread's 32-bit word of four codes is its A fragment; V goes through transposing
// 8x8 loads of byte pairs, which put even dims into rows 0-7 of a fragment and odd
// ones into rows 8-15.
//
// A sequence's run that does not cover it whole leaves a partial result (values,
// reference, sum): the warps of a CTA join theirs in shared memory, CTAs through the
// workspace, where the last to arrive at a sequence joins the records in order.
#pragma once

#include <cfloat>

#include "paged.cuh"

namespace lrkv {
namespace paged {

constexpr int kTile = 32;                // tokens
constexpr int kUnitBytes = kTile * kD;   // codes of a tile's keys, or of its values
// The reference of a row's weights is set 7 below its maximum and moves when the maximum is more
// than 15 above it (log2): weights reach 2^15, the top of f16's range, and its smallest step is
// 2^-31 of the largest one's.  (With the maximum as the reference, weights below 2^-25 became zero
// in the products and still counted in the sum that divides them.)
constexpr float kLift = 7.f, kLazyMax = 15.f, kUnlift = 1.f / 128.f;

struct AttnParams {
  CUtensorMap map_k, map_v;   // codes as rows of 128 bytes; box {128, min(page, 32)}
  lrkv_paged_dims D;
  lrkv_paged_cache C;
  const lrkv_bf16* q;
  lrkv_bf16* out;
  const int32_t* t_q_b;
  const float* slopes;
  const int32_t* first_key;
  const int32_t* prefix_end;
  int* tickets;
  float* recs;
  int layer, t_q, g, row_blocks, per_block;   // query rows per block (before padding)
  int window, page_shift;
  uint32_t hr_mul;   // numbers below 2^31 divided by Hkv row_blocks > 1: umulhi(x, hr_mul) >> hr_shift
  int hr_shift;
  uint32_t g_mul;    // numbers below 2^10 divided by g: x g_mul >> 16
  float row_log2;    // scale * log2(e)
  float cap_unit;    // 1 / (softcap log2(e)): a score in log2 units as tanh's argument (0: no cap)
  float cap_poly[6]; // softcap log2(e) tanh(x) = x (cap_poly[0] + cap_poly[1] x^2 + ..), |x| <= 1
  float cap_log2;    // softcap * log2(e)
};

// A segment is one sequence's tiles for one kv head and row block.  A piece of it that
// one warp has finished, other than the whole of it:
struct Piece {
  int seg;              // number of the segment's first tile; -1: no piece
  int b, hr, tiles;     // sequence, kv head * row blocks + row block, tiles of the segment
};

template <int NB>
struct AttnConfig {
  static constexpr int kWarps = attn_warps(NB), kThreads = 32 * kWarps;
  static constexpr int kUnits = NB == 1 ? 3 : NB == 4 ? 4 : 5;   // ring of a warp, in units
  static constexpr bool kQShared = NB > 1;    // query fragments in shared memory instead of registers
  static constexpr int kQBytes = kQShared ? NB * 2048 : 0;
  static constexpr int kJoin = NB == 1 ? 1 : 4;   // rows that a warp joins side by side
  static constexpr int kRows = 8 * NB, kRec = kRows * kRecFloats;
  static constexpr int kWarpBytes = kUnits * kUnitBytes + kQBytes;
  static_assert(kRec * 4 <= kWarpBytes, "a warp's last record lies in its ring");
  struct Row2 {           // rows 2 t4 and 2 t4 + 1 of an 8-row block
    float s0[2];          // what the sums of keys' products start from
    float mul[2], slope[2], pos[2];
    int lo[2], hi[2];
  };
  struct Shared {
    uint64_t bars[kWarps][kUnits];
    float scale[kWarps][kUnits][2];         // of both halves of a tile (equal with larger pages)
    uint32_t missing[kWarps][kUnits];       // tokens of the tile without a page
    Row2 row[kWarps][NB][4];
    Piece piece[kWarps][2];                 // an early one (workspace), the last one (ring)
    Piece open[2];                          // segments shared with other CTAs: with earlier ones, with later ones alone
    int prefix[kThreads + 1];               // tiles of one kv head before every group of sequences
    int warp_sum[kWarps];
    int abort, last[2], first_cta[2], ctas[2];   // of the open segments
  };
  static constexpr size_t kSmem = (size_t)kWarps * kWarpBytes + sizeof(Shared) + 1024;
};

// What every warp knows of a sequence.
struct Seq {
  int n_rows;    // query rows (tokens) of this call
  int total;     // keys: tokens before and of this call
  int start;     // position of row 0
  int tile0;     // first tile of 32 tokens that some row may see
  int tiles;     // tiles of a segment; 0: no rows
};

__device__ __forceinline__ Seq sequence(const AttnParams& p, int b, uint32_t* status) {
  Seq s;
  const int cap = p.D.max_pages * p.D.page;
  s.n_rows = call_tokens(p.t_q_b, b, p.t_q, status);
  s.start = min(max(p.C.seq_len[b], 0), cap);
  s.total = s.start + s.n_rows;
  if (s.total > cap) *status |= LRKV_DEV_SEQ_OVERFLOW, s.total = cap;
  int lo = 0;
  if (p.window > 0) lo = max(0, s.start - p.window + 1);
  if (p.first_key) {
    int f = 0x7fffffff;
    for (int r = 0; r < s.n_rows; ++r) f = min(f, p.first_key[(size_t)b * p.t_q + r]);
    lo = max(lo, f);
  }
  lo = min(lo, max(s.total - 1, 0));
  s.tile0 = lo / kTile;
  s.tiles = s.n_rows > 0 ? max((s.total + kTile - 1) / kTile - s.tile0, 1) : 0;
  return s;
}

// Where tile number x lies: the sequence, the segment and the tile within it.
struct Place {
  Seq s;
  int b, hr, tile;       // tile: within the segment
  int seg;               // number of the segment's first tile
};

// a / b for 0 <= a < 2^31 and a quotient below 2^20 (kv heads times row blocks: 65535 x 16, or
// 14800 x 64): the fp32 quotient is off by one at most.
__device__ __forceinline__ int div_small(int a, int b, float inv_b) {
  int q = (int)((float)a * inv_b);
  const int r = a - q * b;
  q += r >= b;
  q -= r < 0;
  return q;
}

// The sequences' tiles, so that tile numbers can be looked up: with up to 32 sequences every
// warp holds them in its lanes, else shared memory holds the tiles before every group of
// per_thread sequences (n groups, n + 1 entries, n % 32 == 0).
struct Index {
  const int* prefix;
  int n, per_thread, hr_n;
  Seq mine;       // up to 32 sequences: this lane's
  int before;     // tiles of one kv head and row block before it

  __device__ __forceinline__ Place locate(const AttnParams& p, int x, int lane) const {
    const int unit = hr_n == 1 ? x : (int)(__umulhi((uint32_t)x, p.hr_mul) >> p.hr_shift);
    Place at;
    int first;   // tiles before the sequence
    if (p.D.B <= 32) {   // the last sequence that starts at or before x and is not empty
      at.b = 31 - __clz(__ballot_sync(0xffffffffu, before <= unit && mine.tiles > 0));
      at.s.n_rows = __shfl_sync(0xffffffffu, mine.n_rows, at.b);
      at.s.total = __shfl_sync(0xffffffffu, mine.total, at.b);
      at.s.start = __shfl_sync(0xffffffffu, mine.start, at.b);
      at.s.tile0 = __shfl_sync(0xffffffffu, mine.tile0, at.b);
      at.s.tiles = __shfl_sync(0xffffffffu, mine.tiles, at.b);
      first = __shfl_sync(0xffffffffu, before, at.b) * hr_n;
    } else {
      const int step = n / 32;             // prefix <= x / hr_n  <=>  prefix * hr_n <= x
      const int hi = __popc(__ballot_sync(0xffffffffu, prefix[lane * step] <= unit)) - 1;
      const int lo = __popc(__ballot_sync(0xffffffffu, lane < step && prefix[hi * step + lane] <= unit)) - 1;
      const int group = hi * step + lo;    // the last group that starts at or before x
      at.b = group * per_thread;
      first = prefix[group] * hr_n;
      uint32_t st = 0;
      for (;; ++at.b) {
        at.s = sequence(p, at.b, &st);
        const int all = at.s.tiles * hr_n;
        if (x < first + all || at.b + 1 >= p.D.B) break;
        first += all;
      }
    }
    const int off = x - first, tiles = max(at.s.tiles, 1);
    at.hr = div_small(off, tiles, __fdividef(1.f, (float)tiles));
    at.tile = off - at.hr * tiles;
    at.seg = first + at.hr * tiles;
    return at;
  }
};

// x tiles cut into n equal runs: run i is [start(i), start(i + 1)).  n <= 16 for every SM, below
// 2^12, so that rest * i < n^2 < 2^24 is exact in fp32.
struct Runs {
  int n, quot, rest;
  float inv_n, per_tile;   // 1 / n; runs per tile, nearly
  __device__ __forceinline__ Runs(int x, int runs) : n(runs), quot(x / runs), rest(x - quot * runs) {
    inv_n = __fdividef(1.f, (float)runs);
    per_tile = __fdividef((float)runs, (float)x);
  }
  __device__ __forceinline__ int start(int i) const { return quot * i + div_small(rest * i, n, inv_n); }
  // the run that tile t lies in (x > 0)
  __device__ __forceinline__ int of(int t) const {
    int i = min((int)((float)t * per_tile), n - 1);   // off by one at most
    while (start(i) > t) --i;
    while (i + 1 < n && start(i + 1) <= t) ++i;
    return i;
  }
};

__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// Arrives (once) on `bar` when this thread's cp.async copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// Codes to f16x2 of the word's bytes (0, 1) and (2, 3), exactly; int8 codes as (code + 128) 2^-24:
// a byte with its sign bit flipped is code + 128, and a subnormal f16 with that low byte has
// that value in units of 2^-24.  The sums that such operands enter start from what the
// shift adds to them, with the sign turned.  (Taking the shift off every operand instead,
// by two more instructions per word: 168 against 164 us at 131072 tokens x 32 heads, 182 against
// 174 under the power limit; 89 against 81 us for sixteen sequences of 8K to 16K x 8 heads.  As
// normal numbers, with high byte 0x64, codes would come with 1152 added, at the cost of three
// bits of the sums.)
constexpr float kCodeUnit = 1.f / 16777216.f;   // of int8 codes as operands
template <int CODE>
__device__ __forceinline__ void codes_pairs(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if (CODE == LRKV_CODE_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    h01 = __byte_perm(u, 0u, 0x4140);
    h23 = __byte_perm(u, 0u, 0x4342);
  } else {
    codes_f16<CODE>(w, h01, h23);
  }
}
// The same of the bytes (0, 2) and (1, 3).
template <int CODE>
__device__ __forceinline__ void codes_evenodd(uint32_t w, uint32_t& h02, uint32_t& h13) {
  if (CODE == LRKV_CODE_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    h02 = __byte_perm(u, 0u, 0x4240);
    h13 = __byte_perm(u, 0u, 0x4341);
  } else {
    const uint32_t r = __byte_perm(w, 0, 0x3120);
    h02 = e4m3x2_f16x2(r & 0xffffu);
    h13 = e4m3x2_f16x2(r >> 16);
  }
}

// Brings tiles of one warp's run into its ring: keys, values, keys, values, ...
template <int NB, int PT>
struct Producer {
  using C = AttnConfig<NB>;
  Place at;
  int x, end;
  int rows_at;           // tile that lane 0's rows are of
  int row_a, row_b;      // this lane's tile (rows_at + lane): its first row in the tensor map, and
                         // that of its second half where PT = 16; kNotNeeded, kNoPage
  int a, b;              // of the tile whose keys came last
  int slot;              // ring slot of the next unit
  bool values;           // the next unit holds values
  uint32_t status;
  static constexpr int kNotNeeded = -1, kNoPage = -2;

  __device__ __forceinline__ bool more() const { return values || x < end; }
  __device__ __forceinline__ int row_of(const AttnParams& p, int id, int within) {
    if (id < 0 || id >= p.D.n_pages) {
      status |= LRKV_DEV_BAD_PAGE;
      return kNoPage;
    }
    const unsigned ph = ((unsigned)p.layer * p.D.n_pages + id) * p.D.Hkv + (unsigned)(p.row_blocks == 1 ? at.hr : at.hr / p.row_blocks);
    return (int)((ph << p.page_shift) + within);
  }
  __device__ __forceinline__ void load_rows(const AttnParams& p, int lane) {
    rows_at = at.tile;
    const int pos = (at.s.tile0 + at.tile + lane) * kTile;
    row_a = row_b = kNotNeeded;
    const int* row = p.C.page_table + (size_t)at.b * p.D.max_pages + (pos >> p.page_shift);
    if (at.tile + lane >= at.s.tiles) return;
    if (pos < at.s.total) row_a = row_of(p, row[0], pos & (p.D.page - 1));
    if (PT == 16 && pos + 16 < at.s.total) row_b = row_of(p, row[1], 0);
  }
  // Issues the next unit (all lanes call it).
  __device__ __forceinline__ void issue(const AttnParams& p, typename C::Shared& sh, const Index& index,
                                        unsigned char* ring, int warp, int lane) {
    if (!values) {
      if (at.tile >= at.s.tiles || at.tile - rows_at >= 32) {
        if (at.tile >= at.s.tiles) {
          if (at.hr + 1 < index.hr_n) ++at.hr, at.tile = 0;     // the sequence's next head
          else at = index.locate(p, x, lane);
        }
        load_rows(p, lane);
      }
      a = __shfl_sync(0xffffffffu, row_a, at.tile - rows_at);
      b = PT == 16 ? __shfl_sync(0xffffffffu, row_b, at.tile - rows_at) : kNotNeeded;
    }
    if (elect_one()) {
      unsigned char* dst = ring + slot * kUnitBytes;
      uint64_t* bar = &sh.bars[warp][slot];
      float* sc = sh.scale[warp][slot];
      const CUtensorMap* map = values ? &p.map_v : &p.map_k;
      const float* scales = values ? p.C.scale_v : p.C.scale_k;
      if (PT == 16) {
        sh.missing[warp][slot] = (a < 0 ? 0xffffu : 0u) | (b < 0 ? 0xffff0000u : 0u);
        mbar_arrive_expect_tx(bar, ((a >= 0 ? 1u : 0u) + (b >= 0 ? 1u : 0u)) * (PT * kD));
      } else {
        sh.missing[warp][slot] = a < 0 ? 0xffffffffu : 0u;
        mbar_arrive_expect_tx(bar, a >= 0 ? PT * kD : 0);
      }
      if (a >= 0) {
        tma_load_2d(dst, map, 0, a, bar);
        cp_async4(sc, scales + (a >> p.page_shift));
      } else {
        sc[0] = 0.f;
      }
      if (PT == 16) {
        if (b >= 0) {
          tma_load_2d(dst + 16 * kD, map, 0, b, bar);
          cp_async4(sc + 1, scales + (b >> p.page_shift));
        } else {
          sc[1] = 0.f;
        }
      }
      cp_async_arrive(bar);
    }
    __syncwarp();
    slot = slot + 1 == C::kUnits ? 0 : slot + 1;
    if (values) ++at.tile, ++x;
    values = !values;
  }
};

// d = A(16x16 f16, row) * B(16x8 f16, col) + c.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void ldsm_x4_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t_at(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// Where the row `rho` (token * g + head within the group) of kv head h goes.
__device__ __forceinline__ size_t row_offset(const AttnParams& p, int b, int h, int rho) {
  const int tok = (int)((uint32_t)rho * p.g_mul >> 16);
  return (((size_t)b * p.t_q + tok) * p.D.Hq + h * p.g + (rho - tok * p.g)) * kD;
}

// The place of bit number i of the set bits of a mask.
__device__ __forceinline__ int nth_bit(uint32_t mask, int i) {
  int at = 0;
#pragma unroll
  for (int step = 16; step > 0; step >>= 1) {
    const int below = __popc((mask >> at) & ((1u << step) - 1u));
    if (i >= below) i -= below, at += step;
  }
  return at;
}
// Joins rows row0, row0 + step, .. (up to kJoin of them, below `stop`) of n <= 32 records by a
// warp, four values of a row to a lane: weights 2^(m_i - max m).  Lane i holds record i's
// address.  The rows go side by side: one after the other, the maxima and sums over lanes of
// 32 rows took 22000 clocks.
// (kJoin is 1 where a CTA holds 8 rows: a warp seldom has two, and 4 cost 3 us at 8K tokens.)
template <int kJoin>
__device__ __forceinline__ void join_rows(int n, const float* rec, int rows, int row0, int step, int stop, int lane,
                                          float4 (&o)[kJoin], float (&m)[kJoin], float (&l)[kJoin]) {
  const int cnt = kJoin == 1 ? 1 : min(kJoin, (stop - row0 + step - 1) / step);
  float w[kJoin];
  const float* at = rec + rows * kRecRow + row0;
#pragma unroll
  for (int k = 0; k < kJoin; ++k) {
    w[k] = lane < n && k < cnt ? at[k * step] : -INFINITY;
    l[k] = lane < n && k < cnt ? at[rows + k * step] : 0.f;
    m[k] = w[k];
    o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
#pragma unroll
    for (int k = 0; k < kJoin; ++k) m[k] = fmaxf(m[k], __shfl_xor_sync(0xffffffffu, m[k], s));
#pragma unroll
  for (int k = 0; k < kJoin; ++k) {
    w[k] = ex2(w[k] - (m[k] == -INFINITY ? 0.f : m[k]));   // 0 for lanes past n
    l[k] *= w[k];
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
#pragma unroll
    for (int k = 0; k < kJoin; ++k) l[k] += __shfl_xor_sync(0xffffffffu, l[k], s);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* ri = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(rec), i));
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      if (k >= cnt) break;
      const float wi = __shfl_sync(0xffffffffu, w[k], i);
      const float4 v = *reinterpret_cast<const float4*>(ri + (row0 + k * step) * kRecRow + 4 * lane);
      o[k].x = fmaf(wi, v.x, o[k].x), o[k].y = fmaf(wi, v.y, o[k].y);
      o[k].z = fmaf(wi, v.z, o[k].z), o[k].w = fmaf(wi, v.w, o[k].w);
    }
  }
}
__device__ __forceinline__ void store_row4(lrkv_bf16* dst, const float4& o, float l) {
  const float inv = 1.f / l;   // l = 0: the row saw nothing
  *reinterpret_cast<uint2*>(dst) = l == 0.f ? make_uint2(0u, 0u)
                                            : make_uint2(cvt_bf16x2(o.x * inv, o.y * inv), cvt_bf16x2(o.z * inv, o.w * inv));
}

// NB: blocks of 8 query rows; CODE: LRKV_CODE_*; PT: tokens of a tile on one page (16 or 32);
// MOD: scores are capped or get a bias (code that a plain call would have to skip costs it 1 us).
template <int NB, int CODE, int PT, bool MOD>
__global__ void __launch_bounds__(AttnConfig<NB>::kThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  using C = AttnConfig<NB>;
  constexpr int W = C::kWarps, kJoin = C::kJoin, ROWS = C::kRows, kRec = C::kRec;   // a record: values [ROWS][kRecRow], references, sums
  constexpr bool kInt = CODE == LRKV_CODE_INT8;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // rings first: their units are 1024-aligned
  typename C::Shared& sh = *reinterpret_cast<typename C::Shared*>(sm + W * C::kWarpBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  if (lane == 0) {
    for (int s = 0; s < C::kUnits; ++s) mbar_init(&sh.bars[warp][s], 2);
    fence_mbar_init();
    sh.piece[warp][0].seg = sh.piece[warp][1].seg = -1;
  }
  if (tid == 0) {
    sh.abort = 0;
    sh.open[0].seg = sh.open[1].seg = -1;
    sh.last[0] = sh.last[1] = 0;
    tc5::prefetch_tensormap(&p.map_k);
    tc5::prefetch_tensormap(&p.map_v);
  }
  griddep_wait();
  griddep_launch_dependents();

  Index index;
  index.prefix = sh.prefix;
  index.n = C::kThreads;
  index.per_thread = (p.D.B + C::kThreads - 1) / C::kThreads;
  index.hr_n = p.D.Hkv * p.row_blocks;
  uint32_t status = 0;
  int T;
  {
    int n = 0;
    if (p.D.B <= 32) {
      index.mine.tiles = 0;
      if (lane < p.D.B) index.mine = sequence(p, lane, &status);
      n = index.mine.tiles;
    } else {
      const int b0 = tid * index.per_thread, b1 = min(b0 + index.per_thread, p.D.B);
      for (int b = b0; b < b1; ++b) n += sequence(p, b, &status).tiles;
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    index.before = sum - n;
    T = __shfl_sync(0xffffffffu, sum, 31);
    if (p.D.B > 32) {
      if (lane == 31) sh.warp_sum[warp] = sum;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
      sh.prefix[tid + 1] = before + sum;
      if (tid == 0) sh.prefix[0] = 0;
      __syncthreads();
      T = sh.prefix[C::kThreads];
    }
    if (blockIdx.x != 0 || (p.D.B <= 32 && warp != 0)) status = 0;   // reported once
  }
  T *= index.hr_n;
  const int ctas = min((int)gridDim.x, (T + W - 1) / W);   // a tile per warp at least
  if ((int)blockIdx.x >= ctas) {
    if (status) atomicOr(p.C.dev_status, status);
    return;
  }
  const Runs workers(T, ctas * W);
  unsigned char* ring = sm + warp * C::kWarpBytes;
  uint2* q_sh = reinterpret_cast<uint2*>(ring + C::kUnits * kUnitBytes);

  // Four dims of every k-step of query row rho (zeros past the block's rows).
  auto load_q = [&](const Place& at, int rho, int rho1, int h, uint2 (&w)[8]) {
    if (rho < rho1) {
      const lrkv_bf16* src = p.q + row_offset(p, at.b, h, rho) + 4 * t4;
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint2*>(src + 16 * c);
    }
  };
  Producer<NB, PT> prod;
  prod.x = workers.start(blockIdx.x * W + warp);
  prod.end = workers.start(blockIdx.x * W + warp + 1);
  prod.slot = 0;
  prod.values = false;
  prod.status = 0;
  int x = prod.x;
  const int end = prod.end;
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;
  Place at;
  int in_flight = min(C::kUnits, 2 * (end - x));
  // Waits for the next unit; on a time-out leaves no copy in flight.
  auto wait_unit = [&]() {
    if (!ok) return false;
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(&sh.bars[warp][slot], phase, kWaitIters));
    if (!ok) {
      if (lane == 0) sh.abort = 1;
      for (int i = 1; i < in_flight; ++i) {
        const int s = slot + i;
        mbar_wait_bounded(&sh.bars[warp][s % C::kUnits], phase ^ (s >= C::kUnits), kWaitIters);
      }
    }
    return ok;
  };
  // From a raw product to a score in log2 units; positive and finite: an unseen key stays at -inf,
  // a product of 0 at 0.
  auto factor = [](float scale, float mul) {
    const float f = scale * mul;
    return fminf(fmaxf(kInt ? f * (1.f / kCodeUnit) : f, FLT_MIN), FLT_MAX);
  };
  // The unit has been read: bring the next one into its slot.
  auto next_unit = [&]() {
    slot = slot + 1 == C::kUnits ? 0 : slot + 1;
    phase ^= slot == 0;
    __syncwarp();
    if (prod.more()) prod.issue(p, sh, index, ring, warp, lane);
    else --in_flight;
  };

  for (bool first = true; x < end; first = false) {
    at = index.locate(p, x, lane);
    const int h = p.row_blocks == 1 ? at.hr : at.hr / p.row_blocks, rb = at.hr - h * p.row_blocks;
    const int n_tiles = min(at.s.tiles - at.tile, end - x);
    const int rho0 = rb * p.per_block, rho1 = min(min(rho0 + p.per_block, p.g * p.t_q), p.g * at.s.n_rows);
    uint2 q_next[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) q_next[c] = make_uint2(0u, 0u);
    load_q(at, rho0 + g8, rho1, h, q_next);
    if (first) {   // beside the queries' way
      prod.at = at;
      prod.load_rows(p, lane);
#pragma unroll 1
      for (int s = 0; s < C::kUnits && prod.more(); ++s) prod.issue(p, sh, index, ring, warp, lane);
    }

    // queries of the block as B fragments, scaled by a power of two per row so that the
    // row's largest element lies in [2^14, 2^15): f16 then keeps what is above 2^-28 of it
    uint32_t qf[C::kQShared ? 1 : NB][8][2];
    float m[NB][2], l[NB][2];
    int all_lo = 0, all_hi = 0x7fffffff;   // keys that every row sees
    const uint32_t minus_shift[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};   // f16x2 of -128 units
    __syncwarp();
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) m[nb][0] = m[nb][1] = -INFINITY, l[nb][0] = l[nb][1] = 0.f;
#pragma unroll 1
    for (int nb = 0; nb < NB; ++nb) {
      uint2 w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = q_next[c], q_next[c] = make_uint2(0u, 0u);
      if (nb + 1 < NB) load_q(at, rho0 + 8 * (nb + 1) + g8, rho1, h, q_next);
      uint32_t mag = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) mag = __vmaxu2(mag, __vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu));
      mag = max(mag & 0xffffu, mag >> 16);
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
      const int e = min(max((int)(mag >> 7), 15), 254) - 127;          // 2^e <= largest < 2^(e+1)
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);  // 2^(14 - e), between 2^-113 and 2^126
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t b0 = cvt_f16x2(bf_lo(w[c].x) * up, bf_hi(w[c].x) * up);
        const uint32_t b1 = cvt_f16x2(bf_lo(w[c].y) * up, bf_hi(w[c].y) * up);
        if (kInt) mma_f16(acc, minus_shift, b0, b1, acc);
        if (C::kQShared) q_sh[(c * NB + nb) * 32 + lane] = make_uint2(b0, b1);
        else qf[0][c][0] = b0, qf[0][c][1] = b1;
      }
      // this thread's score columns are rows 2 t4, 2 t4 + 1; lane t4 keeps what is known of them
      typename C::Row2 row;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        row.s0[j] = acc[j];
        const int er = __shfl_sync(0xffffffffu, e, (2 * t4 + j) * 4);
        row.mul[j] = p.row_log2 * __uint_as_float((uint32_t)(127 + er - 14) << 23);   // 2^(e - 14) >= 2^-126
        const int r = rho0 + 8 * nb + 2 * t4 + j;
        row.lo[j] = 0;
        row.hi[j] = 0x7fffffff;
        row.pos[j] = row.slope[j] = 0.f;
        if (r < rho1) {
          const int tok = (int)((uint32_t)r * p.g_mul >> 16);
          const size_t meta = (size_t)at.b * p.t_q + tok;
          const int i = at.s.start + tok;
          int a = p.first_key ? max(p.first_key[meta], 0) : 0, z = i;
          if (p.window > 0) a = max(a, i - p.window + 1);
          if (p.prefix_end) {
            const int e1 = p.prefix_end[meta];
            if (e1 > 0) z = max(z, e1 - 1);
          }
          z = min(z, at.s.total - 1);
          if (a > z) a = 0x7fffffff, z = -1;
          row.lo[j] = a;
          row.hi[j] = z;
          row.pos[j] = (float)i;
          if (MOD && p.slopes) row.slope[j] = p.slopes[h * p.g + r - tok * p.g] * kLog2e;
          all_lo = max(all_lo, a);
          all_hi = min(all_hi, z);
        }
      }
      if (g8 == 0) sh.row[warp][nb][t4] = row;
    }
    __syncwarp();
    all_lo = __reduce_max_sync(0xffffffffu, all_lo);
    all_hi = __reduce_min_sync(0xffffffffu, all_hi);

    float o[NB][8][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int dt = 0; dt < 8; ++dt)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nb][dt][k] = 0.f;

#pragma unroll 1
    for (int it = 0; it < n_tiles; ++it) {
      const int base = (at.s.tile0 + at.tile + it) * kTile;
      if (!wait_unit()) break;   // the results are void, but the joins below still take place
      const uint32_t kt = smem_u32(ring + slot * kUnitBytes) + (lane & 15) * kD + (((lane >> 4) ^ (lane & 7)) << 4);
      const float sk0 = sh.scale[warp][slot][0], sk1 = PT == 16 ? sh.scale[warp][slot][1] : sk0;
      uint32_t gone = sh.missing[warp][slot];   // tokens that are not there
      const int valid = at.s.total - base;
      if (valid < kTile) gone |= valid <= 0 ? 0xffffffffu : 0xffffffffu << valid;

      float s[NB][2][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[nb][mt][k] = kInt ? sh.row[warp][nb][t4].s0[k & 1] : 0.f;
#pragma unroll(C::kQShared ? 1 : 4)
      for (int c = 0; c < 8; c += 2) {
        uint32_t a[2][2][4];   // [16 dims][16 tokens]
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t r[4];
          ldsm_x4_at(r, (kt ^ (c << 4)) + mt * 16 * kD);
          codes_pairs<CODE>(r[0], a[0][mt][0], a[0][mt][2]);
          codes_pairs<CODE>(r[1], a[0][mt][1], a[0][mt][3]);
          codes_pairs<CODE>(r[2], a[1][mt][0], a[1][mt][2]);
          codes_pairs<CODE>(r[3], a[1][mt][1], a[1][mt][3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            uint2 b;
            if (C::kQShared) b = q_sh[((c + i) * NB + nb) * 32 + lane];
            else b = make_uint2(qf[0][C::kQShared ? 0 : c + i][0], qf[0][C::kQShared ? 0 : c + i][1]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
              mma_f16(s[nb][mt], a[i][mt], b.x, b.y, s[nb][mt]);
          }
      }
      next_unit();

      const bool whole = base >= all_lo && base + kTile - 1 <= all_hi && gone == 0;
      // weights are 2^(f s - m): the factor f of raw products is 1 once a modifier has been applied
      float mx[NB][2], f[NB][PT == 16 ? 2 : 1][2];
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const typename C::Row2& row = sh.row[warp][nb][t4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          f[nb][0][j] = factor(sk0, row.mul[j]);
          if (PT == 16) f[nb][PT == 16 ? 1 : 0][j] = factor(sk1, row.mul[j]);
        }
        if (MOD) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float v = s[nb][mt][k] * f[nb][PT == 16 ? mt : 0][k & 1];
              if (p.cap_unit > 0.f) {
                const float x = v * p.cap_unit, t = x * x;
                float r = p.cap_poly[5];
#pragma unroll
                for (int i = 4; i >= 0; --i) r = fmaf(r, t, p.cap_poly[i]);
                v = x * r;
                if (fabsf(x) > 1.f)   // tanh x = 1 - 2 / (1 + e^(2 x)), which cancels near 0
                  v = fmaf(-2.f * p.cap_log2, rcp_fast(1.f + ex2(x * (2.f * kLog2e))), p.cap_log2);
              }
              if (p.slopes) {       // positions are below 2^24: exact in fp32
                const float dist = (float)(base + g8 + mt * 16 + 8 * (k >> 1)) - row.pos[k & 1];
                v = fmaf(-row.slope[k & 1], fabsf(dist), v);
              }
              s[nb][mt][k] = v;
            }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f[nb][0][j] = 1.f;
            if (PT == 16) f[nb][PT == 16 ? 1 : 0][j] = 1.f;
          }
        }
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int tok = mt * 16 + 8 * u + g8;
                if (base + tok < row.lo[j] || base + tok > row.hi[j] || (gone >> tok & 1)) s[nb][mt][2 * u + j] = -INFINITY;
              }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float mx0 = fmaxf(s[nb][0][j], s[nb][0][2 + j]), mx1 = fmaxf(s[nb][1][j], s[nb][1][2 + j]);
          if (PT == 16) mx[nb][j] = fmaxf(mx0 * f[nb][0][j], mx1 * f[nb][PT == 16 ? 1 : 0][j]);
          else mx[nb][j] = fmaxf(mx0, mx1) * f[nb][0][j];
          grow |= mx[nb][j] - m[nb][j] > kLazyMax;   // (m + kLazyMax is rounded where m is large)
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = mx[nb][j];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float m_new = fmaxf(m[nb][j], v - kLift);
            const float r = m_new == -INFINITY ? 1.f : ex2(m[nb][j] - m_new);
            m[nb][j] = m_new;
            l[nb][j] *= r;
#pragma unroll
            for (int dt = 0; dt < 8; ++dt) o[nb][dt][j] *= r, o[nb][dt][2 + j] *= r;
          }
      }
      uint32_t pf[NB][2][2];   // weights as B fragments
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const float ref0 = m[nb][0] == -INFINITY ? 0.f : m[nb][0], ref1 = m[nb][1] == -INFINITY ? 0.f : m[nb][1];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float* fm = f[nb][PT == 16 ? mt : 0];
            const float a = ex2(fmaf(s[nb][mt][2 * u], fm[0], -ref0)), c = ex2(fmaf(s[nb][mt][2 * u + 1], fm[1], -ref1));
            l[nb][0] += a;
            l[nb][1] += c;
            pf[nb][mt][u] = movmatrix_t(cvt_f16x2(a, c));
          }
      }
      // the sums of values' products start from minus what the shift adds to them
      float t0[NB][PT == 16 ? 2 : 1][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          float(&t)[4] = t0[nb][PT == 16 ? mt : 0];
          if (mt == 0 || PT == 16) t[0] = t[1] = t[2] = t[3] = 0.f;
          if (kInt) mma_f16(t, minus_shift, pf[nb][mt][0], pf[nb][mt][1], t);
        }

      if (!wait_unit()) break;
      unsigned char* vt = ring + slot * kUnitBytes;
      // units of the results, to which the sums of weights are brought as well: 2^-7 (so that large
      // values find room for lifted weights), of int8 codes 2^-24
      constexpr float kValue = kInt ? 1.f : kUnlift;
      const float sv0 = sh.scale[warp][slot][0] * kValue, sv1 = PT == 16 ? sh.scale[warp][slot][1] * kValue : sv0;
      if (!kInt && gone) {   // what lies there may be a NaN, which a zero weight keeps: clear those rows
        if (gone >> lane & 1) {
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vt + lane * kD + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t vrow = smem_u32(vt) + lane * kD + ((lane & 7) << 4);
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        uint32_t r[4], a[2][4];
        ldsm_x4_t_at(r, vrow ^ (dt << 4));
        codes_evenodd<CODE>(r[0], a[0][0], a[0][1]);
        codes_evenodd<CODE>(r[1], a[0][2], a[0][3]);
        codes_evenodd<CODE>(r[2], a[1][0], a[1][1]);
        codes_evenodd<CODE>(r[3], a[1][2], a[1][3]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float t[4];
          mma_f16(t, a[0], pf[nb][0][0], pf[nb][0][1], t0[nb][0]);
          if (PT == 16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nb][dt][k] = fmaf(sv0, t[k], o[nb][dt][k]);
            mma_f16(t, a[1], pf[nb][1][0], pf[nb][1][1], t0[nb][PT == 16 ? 1 : 0]);
          } else {
            mma_f16(t, a[1], pf[nb][1][0], pf[nb][1][1], t);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nb][dt][k] = fmaf(sv1, t[k], o[nb][dt][k]);
        }
      }
      next_unit();
    }
    x += n_tiles;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 4);
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 8);
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 16);
        l[nb][j] *= kInt ? kCodeUnit : kUnlift;
      }
    if (at.tile == 0 && n_tiles == at.s.tiles) {   // the whole segment: write it
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = rho0 + 8 * nb + 2 * t4 + j;
          if (r >= rho1) continue;
          const float inv = 1.f / l[nb][j];
          lrkv_bf16* dst = p.out + row_offset(p, at.b, h, r) + 2 * g8;
#pragma unroll
          for (int dt = 0; dt < 8; ++dt)
            *reinterpret_cast<uint32_t*>(dst + 16 * dt) =
                l[nb][j] == 0.f ? 0u : cvt_bf16x2(o[nb][dt][j] * inv, o[nb][dt][2 + j] * inv);
        }
    } else {
      const int late = x < end ? 0 : 1;
      // the last piece goes into the ring (nothing is in flight any more), an early one into the workspace
      float* rec = late ? reinterpret_cast<float*>(ring) : p.recs + ((size_t)blockIdx.x * (2 + W) + 2 + warp) * kRec;
      __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nb + 2 * t4 + j;
#pragma unroll
          for (int dt = 0; dt < 8; ++dt)
            *reinterpret_cast<float2*>(rec + r * kRecRow + 16 * dt + 2 * g8) = make_float2(o[nb][dt][j], o[nb][dt][2 + j]);
          if (g8 == 0) rec[ROWS * kRecRow + r] = m[nb][j], rec[ROWS * kRecRow + ROWS + r] = l[nb][j];
        }
      if (lane == 0) {
        Piece& pc = sh.piece[warp][late];
        pc.seg = at.seg;
        pc.b = at.b;
        pc.hr = at.hr;
        pc.tiles = at.s.tiles;
      }
    }
  }
  status |= prod.status;
  if (status) atomicOr(p.C.dev_status, status);
  __syncthreads();
  if (sh.abort && tid == 0) atomicOr(p.C.dev_status, LRKV_DEV_WAIT_TIMEOUT);

  const int X0 = workers.start(blockIdx.x * W), X1 = workers.start((blockIdx.x + 1) * W);
  auto cta_of = [&](int tile) { return workers.of(tile) / W; };
  // Rounds 0 and 1 join the pieces of a segment that lie in this CTA: the warps that hold them
  // share the rows.  Rounds 2 and 3 join the records of a segment that several CTAs share, where
  // this CTA is the last to arrive: with earlier CTAs, with later ones.  (One copy of the code for
  // all rounds: much of a short call's time goes on fetching instructions for the first time.)
#pragma unroll 1
  for (int round = 0; round < 4; ++round) {
    if (round == 2) {
      __syncthreads();
      if (sh.open[0].seg < 0 && sh.open[1].seg < 0) return;
      if (tid < 2 && sh.open[tid].seg >= 0) {
        const int c0 = cta_of(sh.open[tid].seg), c1 = cta_of(sh.open[tid].seg + sh.open[tid].tiles - 1);
        sh.last[tid] = atom_add_acq_rel_gpu(p.tickets + c0, 1) == c1 - c0;
        if (sh.last[tid]) p.tickets[c0] = 0;
        sh.first_cta[tid] = c0;
        sh.ctas[tid] = c1 - c0 + 1;
      }
      __syncthreads();
    }
    const bool mine = round < 2;
    const Piece pc = mine ? sh.piece[warp][round] : sh.open[round - 2];
    if (pc.seg < 0 || (!mine && !sh.last[round - 2])) continue;
    // query rows of the block
    uint32_t st = 0;
    const int h = p.row_blocks == 1 ? pc.hr : pc.hr / p.row_blocks, rho0 = (pc.hr - h * p.row_blocks) * p.per_block;
    const int rows = min(min(p.per_block, p.g * p.t_q - rho0), p.g * call_tokens(p.t_q_b, pc.b, p.t_q, &st) - rho0);
    int n, row0 = warp, step = W;
    const float* rec = nullptr;
    const bool done = !mine || (pc.seg >= X0 && pc.seg + pc.tiles <= X1);
    const int which = pc.seg >= X0 ? 1 : 0;
    float* dst = p.recs + ((size_t)blockIdx.x * (2 + W) + which) * kRec;
    if (mine) {
      const int seg = lane < 2 * W ? sh.piece[lane >> 1][lane & 1].seg : -1;
      const uint32_t members = __ballot_sync(0xffffffffu, seg == pc.seg);
      step = n = __popc(members);
      row0 = __popc(members & ((1u << (2 * warp + round)) - 1u));
      const int place = nth_bit(members, min(lane, n - 1)), w = place >> 1;
      rec = place & 1 ? reinterpret_cast<const float*>(sm + w * C::kWarpBytes)
                      : p.recs + ((size_t)blockIdx.x * (2 + W) + 2 + w) * kRec;
      if (!done && row0 == 0 && lane == 0) sh.open[which] = pc;
    } else {
      n = sh.ctas[round - 2];
    }
    for (; row0 < rows; row0 += kJoin * step) {
      float4 o[kJoin];
      float m[kJoin], l[kJoin];
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += 32) {   // up to 32 records at a time
        if (!mine) {
          const int i = min(i0 + lane, n - 1);
          rec = p.recs + ((size_t)(sh.first_cta[round - 2] + i) * (2 + W) + (i == 0 ? 1 : 0)) * kRec;
        }
        float4 o1[kJoin];
        float m1[kJoin], l1[kJoin];
        join_rows<kJoin>(min(32, n - i0), rec, ROWS, row0, step, rows, lane, o1, m1, l1);
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
          if (i0 == 0) {
            o[j] = o1[j], m[j] = m1[j], l[j] = l1[j];
            continue;
          }
          const float mm = fmaxf(m[j], m1[j]), ref = mm == -INFINITY ? 0.f : mm;
          const float w = ex2(m[j] - ref), w1 = ex2(m1[j] - ref);
          o[j] = make_float4(o[j].x * w + o1[j].x * w1, o[j].y * w + o1[j].y * w1, o[j].z * w + o1[j].z * w1,
                             o[j].w * w + o1[j].w * w1);
          l[j] = l[j] * w + l1[j] * w1;
          m[j] = mm;
        }
      }
#pragma unroll
      for (int j = 0; j < kJoin; ++j) {
        const int row = row0 + j * step;
        if (row >= rows) continue;
        if (done) {
          store_row4(p.out + row_offset(p, pc.b, h, rho0 + row) + 4 * lane, o[j], l[j]);
        } else {
          *reinterpret_cast<float4*>(dst + row * kRecRow + 4 * lane) = o[j];
          if (lane == 0) dst[ROWS * kRecRow + row] = m[j], dst[ROWS * kRecRow + ROWS + row] = l[j];
        }
      }
    }
  }
}

}  // namespace paged
}  // namespace lrkv
