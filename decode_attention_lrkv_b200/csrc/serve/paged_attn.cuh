// Attention of a few query rows over the pages of the 8-bit cache.
//
// For every query row i of a kv head's group:  o_i = sum_j p_ij s_v(j) c_v,j / sum_j p_ij,
// p_ij = exp(s_ij - m_i), s_ij the modified scores of (q_i . c_k,j) s_k(j), with codes c
// and the scale s of the page that j lies on.
//
// Bound: memory (2 d bytes a token and kv head, read once).  The keys of all
// (sequence, kv head, block of up to 24 query rows) are cut into tiles of 32 tokens
// and numbered; every warp of the grid takes an equal, contiguous run of tiles, so
// ragged lengths, few long sequences and many short ones all fill the SMs alike.
// A warp works alone: its lane 0 brings tiles in by TMA (128-byte swizzle, a ring of
// kStages tiles of keys and values, the scales by 4-byte copies on the same barrier),
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

#include "paged.cuh"

namespace lrkv {
namespace paged {

constexpr int kTile = 32;                    // tokens
constexpr int kStages = 3;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kSideBytes = kTile * kD;       // codes of a tile's keys (or values)
constexpr int kStageBytes = 2 * kSideBytes;
constexpr int kWarpRing = kStages * kStageBytes;
constexpr float kLazyMax = 8.f;              // rescale when a maximum grows by more (log2)

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
  float row_log2;    // scale * log2(e)
  float cap_in;      // 2 / softcap: exponent of e in tanh, per unit of a score (0: no cap)
  float cap_log2;    // softcap * log2(e)
};

// A piece of a sequence's tiles that one warp has finished.
struct Piece {
  long long seg;        // number of the segment's first tile; -1: none
  int b, hr, tiles;     // sequence, kv head * row blocks + row block, tiles of the segment
};

struct AttnShared {
  uint64_t bars[kAttnWarps][kStages];
  float scale[kAttnWarps][kStages][4];       // keys of both halves, values of both halves
  uint32_t missing[kAttnWarps][kStages];     // tokens of the tile without a page
  Piece piece[kAttnWarps][2];                // an early one (workspace), the last one (ring)
  long long prefix[kAttnThreads + 1];        // tiles of one kv head before every group of sequences
  long long warp_sum[kAttnWarps];
  int abort, last[2];
};
inline size_t attn_smem_bytes() { return (size_t)kAttnWarps * kWarpRing + sizeof(AttnShared) + 1024; }

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
  long long seg;         // number of the segment's first tile
};

__device__ __forceinline__ Place locate(const AttnParams& p, const AttnShared& sh, long long x, int per_thread,
                                        int hr_n) {
  int lo = 0, hi = kAttnThreads;   // the last group whose first tile is not behind x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sh.prefix[mid] * hr_n <= x) lo = mid; else hi = mid;
  }
  Place at;
  at.b = lo * per_thread;
  long long before = sh.prefix[lo] * hr_n;
  uint32_t st = 0;
  for (;; ++at.b) {
    at.s = sequence(p, at.b, &st);
    const long long all = (long long)at.s.tiles * hr_n;
    if (x < before + all || at.b + 1 >= p.D.B) break;
    before += all;
  }
  const long long off = x - before, n = max(at.s.tiles, 1);
  at.hr = (int)(off / n);
  at.tile = (int)(off - at.hr * n);
  at.seg = before + at.hr * n;
  return at;
}

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

// Codes to f16x2 of the word's bytes (0, 2) and (1, 3), exactly.
template <int CODE>
__device__ __forceinline__ void codes_evenodd(uint32_t w, uint32_t& h02, uint32_t& h13) {
  if (CODE == LRKV_CODE_INT8) {
    s8x4_f16evenodd(w, h02, h13);
  } else {
    const uint32_t r = __byte_perm(w, 0, 0x3120);
    h02 = e4m3x2_f16x2(r & 0xffffu);
    h13 = e4m3x2_f16x2(r >> 16);
  }
}

// Brings tiles of one warp's run into its ring, one after the other.
template <int PT>
struct Producer {
  Place at;
  long long x, end;
  int ids_at;            // tile that lane 0's ids are of
  int id_a, id_b;        // this lane's page ids (tile ids_at + lane; both halves where PT = 16)
  uint32_t status;

  __device__ __forceinline__ void load_ids(const AttnParams& p, int lane) {
    ids_at = at.tile;
    const int t = at.s.tile0 + at.tile + lane;     // tile of the sequence
    id_a = id_b = -2;                              // not needed
    const size_t row = (size_t)at.b * p.D.max_pages;
    const long long pos = (long long)t * kTile;
    if (pos < at.s.total) id_a = p.C.page_table[row + (size_t)(pos >> p.page_shift)];
    if (PT == 16 && pos + 16 < at.s.total) id_b = p.C.page_table[row + (size_t)(pos >> p.page_shift) + 1];
  }
  __device__ __forceinline__ void begin(const AttnParams& p, const AttnShared& sh, int per_thread, int hr_n, int lane) {
    at = locate(p, sh, x, per_thread, hr_n);
    load_ids(p, lane);
  }
  // Issues the next tile into stage `st` (all lanes call it).
  __device__ __forceinline__ void issue(const AttnParams& p, AttnShared& sh, int per_thread, int hr_n,
                                        unsigned char* ring, int warp, int lane, int st) {
    if (x >= end) return;
    if (at.tile >= at.s.tiles) {
      if (at.hr + 1 < hr_n) {          // the sequence's next head: the same pages
        ++at.hr;
        at.tile = 0;
        if (ids_at != 0) load_ids(p, lane);
      } else {
        begin(p, sh, per_thread, hr_n, lane);
      }
    } else if (at.tile - ids_at >= 32) {
      load_ids(p, lane);
    }
    const int src = at.tile - ids_at;
    const int a = __shfl_sync(0xffffffffu, id_a, src);
    const int b = PT == 16 ? __shfl_sync(0xffffffffu, id_b, src) : -2;
    if (lane == 0) {
      unsigned char* dst = ring + st * kStageBytes;
      uint64_t* bar = &sh.bars[warp][st];
      float* sc = sh.scale[warp][st];
      const int h = at.hr / p.row_blocks;
      const size_t first = (size_t)p.layer * p.D.n_pages;
      uint32_t missing = 0, bytes = 0;
      const bool ok_a = a >= 0 && a < p.D.n_pages, ok_b = PT == 16 && b >= 0 && b < p.D.n_pages;
      if (!ok_a) missing = PT == 16 ? 0xffffu : 0xffffffffu;
      if (PT == 16 && !ok_b) missing |= 0xffff0000u;
      if ((!ok_a && a != -2) || (PT == 16 && !ok_b && b != -2)) status |= LRKV_DEV_BAD_PAGE;
      bytes = ((ok_a ? 1u : 0u) + (ok_b ? 1u : 0u)) * (2u * PT * kD);
      sh.missing[warp][st] = missing;
      mbar_arrive_expect_tx(bar, bytes);
      if (ok_a) {
        const size_t ph = (first + a) * p.D.Hkv + h;
        const int within = PT == 16 ? 0 : ((at.s.tile0 + at.tile) * kTile) & (p.D.page - 1);
        const int y = (int)((ph << p.page_shift) + within);
        tma_load_2d(dst, &p.map_k, 0, y, bar);
        tma_load_2d(dst + kSideBytes, &p.map_v, 0, y, bar);
        cp_async4(sc, p.C.scale_k + ph);
        cp_async4(sc + 2, p.C.scale_v + ph);
      } else {
        sc[0] = sc[2] = 0.f;
      }
      if (PT == 16) {
        if (ok_b) {
          const size_t ph = (first + b) * p.D.Hkv + h;
          const int y = (int)(ph << p.page_shift);
          tma_load_2d(dst + 16 * kD, &p.map_k, 0, y, bar);
          tma_load_2d(dst + kSideBytes + 16 * kD, &p.map_v, 0, y, bar);
          cp_async4(sc + 1, p.C.scale_k + ph);
          cp_async4(sc + 3, p.C.scale_v + ph);
        } else {
          sc[1] = sc[3] = 0.f;
        }
      }
      cp_async_arrive(bar);
    }
    __syncwarp();
    ++at.tile;
    ++x;
  }
};

// Where the row `rho` (token * g + head within the group) of kv head h goes.
__device__ __forceinline__ size_t row_offset(const AttnParams& p, int b, int h, int rho) {
  return (((size_t)b * p.t_q + rho / p.g) * p.D.Hq + h * p.g + rho % p.g) * kD;
}

// Joins n records of one row (m, l and four values from d): weights 2^(m_i - max m).
template <typename Rec>
__device__ __forceinline__ void join_rows(int n, Rec rec, int rows, int row, int d, float4& o, float& m, float& l) {
  m = -INFINITY;
  for (int i = 0; i < n; ++i) m = fmaxf(m, rec(i)[rows * kD + row]);
  const float ref = m == -INFINITY ? 0.f : m;
  l = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* r = rec(i);
    const float w = ex2(r[rows * kD + row] - ref);
    const float4 v = *reinterpret_cast<const float4*>(r + row * kD + d);
    l = fmaf(w, r[rows * kD + rows + row], l);
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
  }
}
__device__ __forceinline__ void store_row4(lrkv_bf16* dst, const float4& o, float l) {
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(dst) = l > 0.f ? make_uint2(cvt_bf16x2(o.x * inv, o.y * inv), cvt_bf16x2(o.z * inv, o.w * inv))
                                           : make_uint2(0u, 0u);
}

// NB: blocks of 8 query rows; CODE: LRKV_CODE_*; PT: tokens of a tile on one page (16 or 32).
template <int NB, int CODE, int PT>
__global__ void __launch_bounds__(kAttnThreads, 1) attn_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  AttnShared& sh = *reinterpret_cast<AttnShared*>(sm + kAttnWarps * kWarpRing);
  constexpr int ROWS = 8 * NB;
  constexpr int kRec = ROWS * kRecFloats;   // floats of a record: values [ROWS][kD], references, sums
  static_assert(kRec * 4 <= kWarpRing, "a warp's last record lies in its ring");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, t4 = lane & 3;
  const int hr_n = p.D.Hkv * p.row_blocks;
  const int per_thread = (p.D.B + kAttnThreads - 1) / kAttnThreads;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&sh.bars[warp][s], 2);
    fence_mbar_init();
    sh.piece[warp][0].seg = sh.piece[warp][1].seg = -1;
  }
  if (tid == 0) {
    sh.abort = 0;
    tc5::prefetch_tensormap(&p.map_k);
    tc5::prefetch_tensormap(&p.map_v);
  }
  griddep_wait();
  griddep_launch_dependents();

  // tiles of one kv head and row block before every thread's sequences
  uint32_t status = 0;
  {
    long long n = 0;
    const int b0 = tid * per_thread, b1 = min(b0 + per_thread, p.D.B);
    for (int b = b0; b < b1; ++b) n += sequence(p, b, &status).tiles;
    if (blockIdx.x != 0) status = 0;   // one CTA reports
    long long sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    sh.prefix[tid + 1] = before + sum;
    if (tid == 0) sh.prefix[0] = 0;
    __syncthreads();
  }
  const long long T = sh.prefix[kAttnThreads] * hr_n;
  const long long ctas = min((long long)gridDim.x, (T + kAttnWarps - 1) / kAttnWarps);   // a tile per warp at least
  if (blockIdx.x >= ctas) {
    if (status) atomicOr(p.C.dev_status, status);
    return;
  }
  const long long X0 = T * blockIdx.x / ctas, X1 = T * (blockIdx.x + 1) / ctas;
  const long long worker = (long long)blockIdx.x * kAttnWarps + warp, workers = ctas * kAttnWarps;
  unsigned char* ring = sm + warp * kWarpRing;

  Producer<PT> prod;
  prod.x = T * worker / workers;
  prod.end = T * (worker + 1) / workers;
  prod.status = 0;
  long long x = prod.x;
  const long long end = prod.end;
  int issued = 0, used = 0;
  bool ok = true;
  if (x < end) {
    prod.begin(p, sh, per_thread, hr_n, lane);
#pragma unroll 1
    for (int s = 0; s < kStages && prod.x < end; ++s, ++issued)
      prod.issue(p, sh, per_thread, hr_n, ring, warp, lane, s);
  }

  while (x < end) {
    const Place at = locate(p, sh, x, per_thread, hr_n);
    const int h = at.hr / p.row_blocks, rb = at.hr % p.row_blocks;
    const int n_tiles = (int)min((long long)(at.s.tiles - at.tile), end - x);
    const int rho0 = rb * p.per_block, rho1 = min(min(rho0 + p.per_block, p.g * p.t_q), p.g * at.s.n_rows);

    // queries of the block as B fragments, scaled by a power of two per row so that the
    // row's largest element lies in [2^14, 2^15): f16 then keeps what is above 2^-28 of it
    uint32_t qf[NB][8][2];
    float mul[NB][2], m[NB][2], l[NB][2], slope[NB][2];
    int lo[NB][2], hi[NB][2], pos[NB][2];
    int all_lo = 0, all_hi = 0x7fffffff;   // keys that every row sees
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int rho = rho0 + 8 * nb + g8;
      uint2 w[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) w[c] = make_uint2(0u, 0u);
      if (rho < rho1) {
        const lrkv_bf16* src = p.q + row_offset(p, at.b, h, rho) + 4 * t4;
#pragma unroll
        for (int c = 0; c < 8; ++c) w[c] = *reinterpret_cast<const uint2*>(src + 16 * c);
      }
      uint32_t mag = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) mag = __vmaxu2(mag, __vmaxu2(w[c].x & 0x7fff7fffu, w[c].y & 0x7fff7fffu));
      mag = max(mag & 0xffffu, mag >> 16);
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
      const int e = min(max((int)(mag >> 7), 15), 254) - 127;          // 2^e <= largest < 2^(e+1)
      // 2^(14 - e) as two factors that are normal in fp32
      const int up = 14 - e, up_a = up / 2;
      const float fa = __uint_as_float((uint32_t)(127 + up_a) << 23), fb = __uint_as_float((uint32_t)(127 + up - up_a) << 23);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        qf[nb][c][0] = cvt_f16x2(bf_lo(w[c].x) * fa * fb, bf_hi(w[c].x) * fa * fb);
        qf[nb][c][1] = cvt_f16x2(bf_lo(w[c].y) * fa * fb, bf_hi(w[c].y) * fa * fb);
      }
      // this thread's score columns are rows 2 t4, 2 t4 + 1: their exponents come from lanes of those rows
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int er = __shfl_sync(0xffffffffu, e, (2 * t4 + j) * 4);
        const int down = er - 14, da = down / 2;
        mul[nb][j] = p.row_log2 * __uint_as_float((uint32_t)(127 + da) << 23) * __uint_as_float((uint32_t)(127 + down - da) << 23);
        const int r = rho0 + 8 * nb + 2 * t4 + j;
        m[nb][j] = -INFINITY;
        l[nb][j] = 0.f;
        lo[nb][j] = 0;
        hi[nb][j] = 0x7fffffff;
        pos[nb][j] = 0;
        slope[nb][j] = 0.f;
        if (r < rho1) {
          const int tok = r / p.g;
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
          lo[nb][j] = a;
          hi[nb][j] = z;
          pos[nb][j] = i;
          if (p.slopes) slope[nb][j] = p.slopes[h * p.g + r % p.g] * kLog2e;
          all_lo = max(all_lo, a);
          all_hi = min(all_hi, z);
        }
      }
    }
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
    for (int it = 0; it < n_tiles && ok; ++it) {
      const int st = used % kStages;
      const int base = (at.s.tile0 + at.tile + it) * kTile;
      bool got = mbar_wait_bounded(&sh.bars[warp][st], (used / kStages) & 1, kWaitIters);
      got = __all_sync(0xffffffffu, got);
      if (!got) {   // the results are void, but the joins below still take place
        ok = false;
        if (lane == 0) sh.abort = 1;
        for (int i = used + 1; i < issued; ++i)   // leave no copy in flight
          mbar_wait_bounded(&sh.bars[warp][i % kStages], (i / kStages) & 1, kWaitIters);
        break;
      }
      unsigned char* kt = ring + st * kStageBytes;
      unsigned char* vt = kt + kSideBytes;
      const float sk0 = sh.scale[warp][st][0], sk1 = PT == 16 ? sh.scale[warp][st][1] : sk0;
      const float sv0 = sh.scale[warp][st][2], sv1 = PT == 16 ? sh.scale[warp][st][3] : sv0;
      uint32_t gone = sh.missing[warp][st];
      const int valid = at.s.total - base;
      if (valid < kTile) gone |= valid <= 0 ? 0xffffffffu : 0xffffffffu << valid;
      if (gone) {   // what lies there may be NaN, which a zero weight keeps: clear those value rows
        if (gone >> lane & 1) {
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vt + lane * kD + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }

      float s[NB][2][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[nb][mt][k] = 0.f;
#pragma unroll
      for (int c = 0; c < 8; c += 2)
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int row = mt * 16 + (lane & 15);
          uint32_t r[4], a[2][4];
          ldsm_x4(r[0], r[1], r[2], r[3], kt + row * kD + (((c + (lane >> 4)) ^ (row & 7)) << 4));
          codes_f16<CODE>(r[0], a[0][0], a[0][2]);
          codes_f16<CODE>(r[1], a[0][1], a[0][3]);
          codes_f16<CODE>(r[2], a[1][0], a[1][2]);
          codes_f16<CODE>(r[3], a[1][1], a[1][3]);
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              mma_16816_f16(s[nb][mt], a[i][0], a[i][1], a[i][2], a[i][3], qf[nb][c + i][0], qf[nb][c + i][1]);
        }

      const bool whole = base >= all_lo && base + kTile - 1 <= all_hi && gone == 0;
      float mx[NB][2];
      bool grow = false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f0 = sk0 * mul[nb][j], f1 = PT == 16 ? sk1 * mul[nb][j] : f0;
          mx[nb][j] = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              float v = s[nb][mt][2 * u + j] * (mt ? f1 : f0);
              const int tok = mt * 16 + 8 * u + g8, key = base + tok;
              if (p.cap_in > 0.f)   // softcap tanh(x / softcap) = softcap (1 - 2 / (1 + e^(2 x / softcap)))
                v = fmaf(-2.f * p.cap_log2, rcp_fast(1.f + ex2(v * p.cap_in)), p.cap_log2);
              if (p.slopes) v = fmaf(-slope[nb][j], fabsf((float)(key - pos[nb][j])), v);
              if (!whole && (key < lo[nb][j] || key > hi[nb][j] || (gone >> tok & 1))) v = -INFINITY;
              s[nb][mt][2 * u + j] = v;
              mx[nb][j] = fmaxf(mx[nb][j], v);
            }
          grow |= mx[nb][j] > m[nb][j] + kLazyMax;
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
            const float m_new = fmaxf(m[nb][j], v);
            const float f = m_new == -INFINITY ? 1.f : ex2(m[nb][j] - m_new);
            m[nb][j] = m_new;
            l[nb][j] *= f;
#pragma unroll
            for (int dt = 0; dt < 8; ++dt) o[nb][dt][j] *= f, o[nb][dt][2 + j] *= f;
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
            const float a = ex2(s[nb][mt][2 * u] - ref0), c = ex2(s[nb][mt][2 * u + 1] - ref1);
            l[nb][0] += a;
            l[nb][1] += c;
            pf[nb][mt][u] = movmatrix_t(cvt_f16x2(a, c));
          }
      }
#pragma unroll
      for (int dt = 0; dt < 8; ++dt) {
        uint32_t r[4], a[2][4];
        ldsm_x4_t(r[0], r[1], r[2], r[3], vt + lane * kD + ((dt ^ (lane & 7)) << 4));
        codes_evenodd<CODE>(r[0], a[0][0], a[0][1]);
        codes_evenodd<CODE>(r[1], a[0][2], a[0][3]);
        codes_evenodd<CODE>(r[2], a[1][0], a[1][1]);
        codes_evenodd<CODE>(r[3], a[1][2], a[1][3]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float t[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816_f16(t, a[0][0], a[0][1], a[0][2], a[0][3], pf[nb][0][0], pf[nb][0][1]);
          if (PT == 16) {
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nb][dt][k] = fmaf(sv0, t[k], o[nb][dt][k]), t[k] = 0.f;
          }
          mma_16816_f16(t, a[1][0], a[1][1], a[1][2], a[1][3], pf[nb][1][0], pf[nb][1][1]);
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nb][dt][k] = fmaf(sv1, t[k], o[nb][dt][k]);
        }
      }
      ++used;
      __syncwarp();   // the stage is free
      if (prod.x < end) {
        prod.issue(p, sh, per_thread, hr_n, ring, warp, lane, st);
        ++issued;
      }
    }
    x += n_tiles;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 4);
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 8);
        l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], 16);
      }
    if (at.tile == 0 && n_tiles == at.s.tiles) {   // the whole sequence: write it
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = rho0 + 8 * nb + 2 * t4 + j;
          if (r >= rho1) continue;
          const float inv = l[nb][j] > 0.f ? 1.f / l[nb][j] : 0.f;
          lrkv_bf16* dst = p.out + row_offset(p, at.b, h, r) + 2 * g8;
#pragma unroll
          for (int dt = 0; dt < 8; ++dt)
            *reinterpret_cast<uint32_t*>(dst + 16 * dt) =
                l[nb][j] > 0.f ? cvt_bf16x2(o[nb][dt][j] * inv, o[nb][dt][2 + j] * inv) : 0u;
        }
    } else {
      const int slot = x < end ? 0 : 1;
      // the last piece goes into the ring (nothing is in flight any more), an early one into the workspace
      float* rec = slot ? reinterpret_cast<float*>(ring)
                        : p.recs + ((size_t)blockIdx.x * (2 + kAttnWarps) + 2 + warp) * kRec;
      __syncwarp();
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = 8 * nb + 2 * t4 + j;
#pragma unroll
          for (int dt = 0; dt < 8; ++dt)
            *reinterpret_cast<float2*>(rec + r * kD + 16 * dt + 2 * g8) = make_float2(o[nb][dt][j], o[nb][dt][2 + j]);
          if (g8 == 0) rec[ROWS * kD + r] = m[nb][j], rec[ROWS * kD + ROWS + r] = l[nb][j];
        }
      if (lane == 0) {
        Piece& pc = sh.piece[warp][slot];
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

  // join the warps' pieces, sequence by sequence
  bool shared_rec[2] = {false, false};
  Piece shared_piece[2];
  for (int i = 0; i < 2 * kAttnWarps;) {
    const Piece first = sh.piece[i >> 1][i & 1];
    if (first.seg < 0) {
      ++i;
      continue;
    }
    int idx[2 * kAttnWarps], n = 0;
    for (; i < 2 * kAttnWarps; ++i) {
      const long long seg = sh.piece[i >> 1][i & 1].seg;
      if (seg < 0) continue;
      if (seg != first.seg) break;
      idx[n++] = i;
    }
    auto rec = [&](int k) -> const float* {
      const int w = idx[k] >> 1;
      return idx[k] & 1 ? reinterpret_cast<const float*>(sm + w * kWarpRing)
                        : p.recs + ((size_t)blockIdx.x * (2 + kAttnWarps) + 2 + w) * kRec;
    };
    const int h = first.hr / p.row_blocks, rho0 = first.hr % p.row_blocks * p.per_block;
    uint32_t st = 0;
    const int rows_b = p.g * call_tokens(p.t_q_b, first.b, p.t_q, &st);
    const int rho1 = min(min(rho0 + p.per_block, p.g * p.t_q), rows_b);
    const bool done = first.seg >= X0 && first.seg + first.tiles <= X1;
    const int which = first.seg >= X0 ? 1 : 0;
    float* dst = p.recs + ((size_t)blockIdx.x * (2 + kAttnWarps) + which) * kRec;
    for (int e = tid; e < ROWS * (kD / 4); e += kAttnThreads) {
      const int row = e / (kD / 4), d = e % (kD / 4) * 4;
      if (rho0 + row >= rho1) continue;
      float4 o;
      float m, l;
      join_rows(n, rec, ROWS, row, d, o, m, l);
      if (done) {
        store_row4(p.out + row_offset(p, first.b, h, rho0 + row) + d, o, l);
      } else {
        *reinterpret_cast<float4*>(dst + row * kD + d) = o;
        if (d == 0) dst[ROWS * kD + row] = m, dst[ROWS * kD + ROWS + row] = l;
      }
    }
    if (!done) {
      if (which) shared_rec[1] = true, shared_piece[1] = first;
      else shared_rec[0] = true, shared_piece[0] = first;
    }
  }
  if (!shared_rec[0] && !shared_rec[1]) return;
  __syncthreads();
  auto cta_of = [&](long long tile) { return (int)(((tile + 1) * ctas + T - 1) / T - 1); };
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      sh.last[k] = 0;
      if (!shared_rec[k]) continue;
      const int c0 = cta_of(shared_piece[k].seg), c1 = cta_of(shared_piece[k].seg + shared_piece[k].tiles - 1);
      if (atom_add_acq_rel_gpu(p.tickets + c0, 1) == c1 - c0) {
        p.tickets[c0] = 0;
        sh.last[k] = 1;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!shared_rec[k] || !sh.last[k]) continue;
    const Piece first = shared_piece[k];
    const int c0 = cta_of(first.seg), c1 = cta_of(first.seg + first.tiles - 1);
    auto rec = [&](int i) -> const float* {
      return p.recs + ((size_t)(c0 + i) * (2 + kAttnWarps) + (i == 0 ? 1 : 0)) * kRec;
    };
    const int h = first.hr / p.row_blocks, rho0 = first.hr % p.row_blocks * p.per_block;
    uint32_t st = 0;
    const int rows_b = p.g * call_tokens(p.t_q_b, first.b, p.t_q, &st);
    const int rho1 = min(min(rho0 + p.per_block, p.g * p.t_q), rows_b);
    for (int e = tid; e < ROWS * (kD / 4); e += kAttnThreads) {
      const int row = e / (kD / 4), d = e % (kD / 4) * 4;
      if (rho0 + row >= rho1) continue;
      float4 o;
      float m, l;
      join_rows(c1 - c0 + 1, rec, ROWS, row, d, o, m, l);
      store_row4(p.out + row_offset(p, first.b, h, rho0 + row) + d, o, l);
    }
  }
}

}  // namespace paged
}  // namespace lrkv
