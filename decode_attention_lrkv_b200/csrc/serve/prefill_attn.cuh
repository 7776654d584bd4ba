// Prefill attention on the 5th-generation tensor cores.
//
// For every query row i of a head:  o_i = sum_j p_ij v_j / sum_j p_ij,
// p_ij = exp(s_ij - m_i), s_ij the modified scores (lrkv_score), m_i a running
// reference close to the row's maximum; one pass over the keys in units of 64.
//
// A CTA takes two blocks of 128 query rows (X = 0, 1) of one head.  Per unit and block:
//     S_X = Q_X K^T      (M 128, N 64, K 128; operands in shared memory)
//     P_X = exp2(S_X ..) (a thread per row; P_X overwrites S_X as packed bf16)
//     O_X += P_X V       (M 128, N 128, K 64; P_X read from tensor memory)
// A block's scores have two places of 64 columns, for even and odd units: with
// O_0, O_1 they fill the 512 columns of tensor memory.  One warp issues TMA loads
// (128-byte swizzle, rings of key and value units), two issue the MMAs of a block
// each, two groups of four warps do the softmax of a block each.  When a block's P of
// unit u arrives its MMA warp issues O += P V of u and S of unit u + 2, so the group
// finds the scores of u + 1 ready: the tensor cores run beside the softmax of the same
// block, not only of the other one.  (One MMA warp for both blocks: 689 us where 511
// had been with units of 128 keys; it spent 1200 clocks a unit on its four waits.)
//
// Bound: a unit of both blocks costs 2 x 2 x 2 x 128 x 64 x 128 tensor flops and
// 2 x 128 x 64 exponentials; at 8192 flops and 16 exponentials a clock and SM both take
// 1024 clocks (1148 measured for the products: S with N = 64 reads shared memory at
// 48 clocks per step where 32 would do).  A unit of both blocks takes 1700 clocks, and a
// CTA 11000 more before its first and after its last one.  8192 causal tokens x 32 heads:
// 466 us (1180 TFLOP/s) at first, 522 to 545 us once the power limit has lowered the clock.
// Also measured, each at first / under the power limit: the softmax groups taking their
// exponentials in turn, one thread issuing all of a block's MMAs, 473 / 578 us; tiles of
// 128 keys, whose S waits for O += P V of the tile before, 511 / 572; those with P in two
// halves, 526 / 586; a quarter or half of the exponentials by a cubic polynomial, which is
// 10 clocks of work on the fp32 pipe against 8 on the special-function unit, no faster.  One
// row block per CTA and two CTAs to an SM, which loads keys and values twice, takes the same
// time here (465 against 466 us, 519 against 522) and more with documents (268 against 257).
//
// The running reference m only moves when a row's maximum passes it by more than
// 2^24 (bf16 and fp32 weights up to 2^24 are as exact as others): O is rescaled in tensor
// memory once or never per row instead of once per unit.  The group that does
// it first waits for the scores of the next unit: MMAs complete in order, so the last
// product into O is complete, and the next one waits for this group's P.
//
// Every mask is an interval [lo, hi] of keys per row, so a block's units are the
// union of its rows' intervals, and a unit inside all of a warp's intervals is not
// masked at all.
#pragma once

#include <cuda.h>

#include "../lrkv_common.cuh"
#include "../tc_ptx.cuh"
#include "lrkv_serve.h"
#include "serve_ptx.cuh"

namespace lrkv {
namespace prefill {

using namespace serve;

constexpr int kTile = 128;                  // query rows per block
constexpr int kUnit = 64;                   // keys per unit
constexpr int kThreads = 352;               // warps 0-3, 4-7 softmax of block 0, 1; 8 TMA; 9, 10 MMA of block 0, 1
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kTileBytes = kTile * kD * 2;  // two boxes of 64 columns
constexpr int kBoxBytes = kTileBytes / 2;
constexpr int kUnitBytes = kUnit * kD * 2;  // two boxes of 64 columns
constexpr int kUnitBox = kUnitBytes / 2;
constexpr int kKStages = 4, kVStages = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 X (+ 64 (unit & 1) for S)
constexpr float kLazy = 24.f;               // rescale when a maximum grows by more (log2)

// Shared memory: Q blocks, key ring, value ring (each 1024-aligned), barriers.
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kKStages * kUnitBytes;
constexpr int kOffBar = kOffV + kVStages * kUnitBytes;
constexpr size_t kSmemBytes = kOffBar + 256 + 1024;

struct Params {
  CUtensorMap map_q, map_k, map_v;   // [B][t][H][128] as (128, H, t, B), box {64, 1, 64, 1}
  lrkv_bf16* out;
  int64_t os_b, os_t, os_h;
  const int32_t* q_len;
  const int32_t* kv_len;
  uint32_t* dev_status;
  const float* slopes;
  const int32_t* first_key;
  const int32_t* prefix_end;
  int B, Hq, Hkv, t_q, t_k, window;
  int n_blocks;       // pairs of query blocks per (b, head)
  float qk_log2;      // scale * log2(e)
  float cap_unit;     // scale / softcap
  float cap_in;       // 2 log2(e) scale / softcap
  float cap_log2;     // softcap * log2(e)
  float cap_poly[6];  // softcap log2(e) tanh(x) = x (cap_poly[0] + cap_poly[1] x^2 + ..), |x| <= 1
  int out32;          // 32-byte stores allowed
  int n_split;        // CTAs that share a pair of query blocks' keys
  float* part;        // n_split > 1: [n_split][B][Hq][t_q][kPart] results before the join
};
// A row's result of one split: O (not divided), the reference, the sum.
constexpr int kPart = kD + 4;

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], p_full[2][2];   // [block][unit & 1]
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int lo[2], hi[2];    // union of the rows' key intervals, per block
};
static_assert(sizeof(Bars) <= 256, "barrier region");

// s[c] = softcap log2(e) tanh(scale s[c] / softcap).  Where all |x| = |scale s / softcap| of
// the warp are at most 1, as sane logits are, by a polynomial in x^2 on the two-wide fp32
// pipe (relative error 6.5e-7: at most 4e-5 in the exponent at softcap 50); else by
// tanh(x) = 1 - 2 / (1 + e^(2x)), two special-function results for each score.
__device__ __forceinline__ void cap_scores(const Params& p, float (&s)[kUnit]) {
  float top0 = 0.f, top1 = 0.f;
#pragma unroll
  for (int c = 0; c < kUnit; c += 4) {
    top0 = max3(top0, fabsf(s[c]), fabsf(s[c + 1]));
    top1 = max3(top1, fabsf(s[c + 2]), fabsf(s[c + 3]));
  }
  // scores of keys past the sequence may be NaN, which a maximum drops; they are masked later
  if (__all_sync(0xffffffffu, fmaxf(top0, top1) * p.cap_unit <= 1.f)) {
    const f32x2 u = pack2(p.cap_unit, p.cap_unit);
    f32x2 k[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) k[i] = pack2(p.cap_poly[i], p.cap_poly[i]);
#pragma unroll
    for (int c = 0; c < kUnit; c += 2) {
      const f32x2 x = mul2(pack2(s[c], s[c + 1]), u), t = mul2(x, x);
      f32x2 r = fma2(k[5], t, k[4]);
      r = fma2(r, t, k[3]);
      r = fma2(r, t, k[2]);
      r = fma2(r, t, k[1]);
      r = fma2(r, t, k[0]);
      unpack2(mul2(x, r), s[c], s[c + 1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < kUnit; ++c) s[c] = fmaf(-2.f * p.cap_log2, rcp_fast(1.f + ex2(s[c] * p.cap_in)), p.cap_log2);
  }
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(sm + kOffBar);
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  griddep_wait();
  griddep_launch_dependents();
  // the last query blocks first: under a causal mask they are the longest
  const int split = blockIdx.x % p.n_split, cta = blockIdx.x / p.n_split;
  const int hb = cta % (p.Hq * p.B);
  const int h = hb % p.Hq, b = hb / p.Hq;
  const int blk = p.n_blocks - 1 - cta / (p.Hq * p.B);
  const int hk = h / (p.Hq / p.Hkv);
  int n_k = p.t_k, n_q = p.t_q;
  uint32_t bad = 0;
  if (p.kv_len) {
    n_k = p.kv_len[b];
    if (n_k < 0 || n_k > p.t_k) bad = LRKV_DEV_BAD_COUNT, n_k = n_k < 0 ? 0 : p.t_k;
  }
  if (p.q_len) {
    n_q = p.q_len[b];
    if (n_q < 0 || n_q > p.t_q) bad = LRKV_DEV_BAD_COUNT, n_q = n_q < 0 ? 0 : p.t_q;
  }
  if (bad && p.dev_status && tid == 0 && blk == 0 && h == 0 && split == 0) atomicOr(p.dev_status, bad);
  const int row0 = blk * 2 * kTile;
  if (row0 >= n_q) return;

  if (tid == 0) {
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < kKStages; ++s) mbar_init(&bars->k_full[s], 1), mbar_init(&bars->k_empty[s], 2);
    for (int s = 0; s < kVStages; ++s) mbar_init(&bars->v_full[s], 1), mbar_init(&bars->v_empty[s], 2);
    for (int x = 0; x < 2; ++x) {
      for (int i = 0; i < 2; ++i) mbar_init(&bars->s_full[x][i], 1), mbar_init(&bars->p_full[x][i], kTile);
      bars->lo[x] = 0x7fffffff;
      bars->hi[x] = -1;
    }
    mbar_init(&bars->drain, 2);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc5::tmem_alloc(&bars->tmem, kTmemCols);
    tc5::tmem_relinquish();
  }
  if (warp == kTmaWarp && lane == 0) {
    tc5::prefetch_tensormap(&p.map_q);
    tc5::prefetch_tensormap(&p.map_k);
    tc5::prefetch_tensormap(&p.map_v);
  }
  __syncthreads();
  // this thread's row (softmax warps): position and key interval
  const int row = row0 + tid;
  int pos = 0, lo = 0x7fffffff, hi = -1;
  if (warp < 8) {
    pos = n_k - n_q + row;
    if (row < n_q) {
      const size_t at = (size_t)b * p.t_q + row;
      lo = p.first_key ? p.first_key[at] : 0;
      if (lo < 0) lo = 0;
      if (p.window > 0 && pos - p.window + 1 > lo) lo = pos - p.window + 1;
      hi = pos;
      if (p.prefix_end) {
        const int e = p.prefix_end[at];
        if (e > 0 && e - 1 > hi) hi = e - 1;
      }
      if (hi > n_k - 1) hi = n_k - 1;
      if (lo > hi) lo = 0x7fffffff, hi = -1;
    }
    const int wlo = __reduce_min_sync(0xffffffffu, lo), whi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
      atomicMin(&bars->lo[warp >> 2], wlo);
      atomicMax(&bars->hi[warp >> 2], whi);
    }
  }
  tc5::fence_before_sync();
  __syncthreads();
  tc5::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem, 0);
  // units [t0[x], t1[x]) of block x; [j0, j1) of the CTA
  int t0[2], t1[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const bool any = bars->hi[x] >= 0;
    t0[x] = __shfl_sync(0xffffffffu, any ? bars->lo[x] / kUnit : 0x7ffffff0, 0);   // known to be uniform
    t1[x] = __shfl_sync(0xffffffffu, any ? bars->hi[x] / kUnit + 1 : 0, 0);
  }
  if (p.n_split > 1) {   // this CTA's share of the units
    const int first = min(t0[0], t0[1]), end = max(t1[0], t1[1]);
    const int per = end > first ? (end - first + p.n_split - 1) / p.n_split : 0;
    const int lo_u = first + split * per, hi_u = lo_u + per;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      t0[x] = max(t0[x], lo_u), t1[x] = min(t1[x], hi_u);
      if (t0[x] >= t1[x]) t0[x] = 0x7ffffff0, t1[x] = 0;
    }
  }
  // The units are taken from the last one down, the nearest keys first: with a distance bias a
  // row then has its maximum at once.  Upwards the reference of a steep head moves in every unit
  // (32 heads, bias over 16384 keys: 2212 us upwards, 1750 down).  From here on units are numbered
  // in the order they are taken.
  const int j0 = min(t0[0], t0[1]), j1 = max(t1[0], t1[1]), top = j0 + j1 - 1;
  auto first_key_of = [&](int j) { return (top - j) * kUnit; };
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (t0[x] < t1[x]) {
      const int last = t1[x] - 1;
      t1[x] = top - t0[x] + 1;
      t0[x] = top - last;
    }

  if (warp == kTmaWarp) {
    if (lane == 0 && j0 < j1) {
      mbar_arrive_expect_tx(&bars->q_full, 2 * kTileBytes);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            tma_load_4d(sm + kOffQ + x * kTileBytes + c * kBoxBytes + r * kUnitBox, &p.map_q, 64 * c, h,
                        row0 + x * kTile + r * kUnit, b, &bars->q_full);
      auto load = [&](const CUtensorMap* map, uint64_t* full, uint64_t* empty, int off, int ns, int j) {
        const int i = j - j0, s = i % ns;
        if (i >= ns && !wait_or_abort(&empty[s], ((i / ns) - 1) & 1, abort_flag)) return false;
        mbar_arrive_expect_tx(&full[s], kUnitBytes);
        unsigned char* dst = sm + off + s * kUnitBytes;
        tma_load_4d(dst, map, 0, hk, first_key_of(j), b, &full[s]);
        tma_load_4d(dst + kUnitBox, map, 64, hk, first_key_of(j), b, &full[s]);
        return true;
      };
      int nk = 0, nv = 0;   // units loaded
      bool ok = true;
      for (int j = j0 - 2; ok && j < j1; ++j) {
        if (j + 2 < j1) {
          ok = load(&p.map_k, bars->k_full, bars->k_empty, kOffK, kKStages, j + 2);
          if (!ok) break;
          ++nk;
        }
        if (j < j0) continue;
        ok = load(&p.map_v, bars->v_full, bars->v_empty, kOffV, kVStages, j);
        if (ok) ++nv;
      }
      // leave no copy in flight: wait for the last fill of every stage
      mbar_wait_bounded(&bars->q_full, 0, kWaitIters);
      for (int i = nk > kKStages ? nk - kKStages : 0; i < nk; ++i)
        mbar_wait_bounded(&bars->k_full[i % kKStages], (i / kKStages) & 1, kWaitIters);
      for (int i = nv > kVStages ? nv - kVStages : 0; i < nv; ++i)
        mbar_wait_bounded(&bars->v_full[i % kVStages], (i / kVStages) & 1, kWaitIters);
    }
  } else if (warp >= kMmaWarp) {
    if (j0 < j1) {
      const int x = warp - kMmaWarp, first = x ? t0[1] : t0[0], end = x ? t1[1] : t1[0];
      constexpr uint32_t idesc_s = tc5::idesc_bf16_f32(kTile, kUnit);
      constexpr uint32_t idesc_o = idesc_bf16_f32_bt(kTile, kD);
      const uint32_t ts = tmem + kColS + 128 * x, to = tmem + kColO + 128 * x;
      // descriptors of the first operands; an offset in shared memory adds its sixteenths
      const uint64_t dq = tc5::smem_desc(smem_u32(sm + kOffQ + x * kTileBytes), 16, 1024, tc5::kSwizzle128B);
      const uint64_t dk = tc5::smem_desc(smem_u32(sm + kOffK), 16, 1024, tc5::kSwizzle128B);
      const uint64_t dv = tc5::smem_desc(smem_u32(sm + kOffV), kUnitBox, 1024, tc5::kSwizzle128B);
      bool ok = wait_or_abort(&bars->q_full, 0, abort_flag);
      for (int j = j0 - 2; j < j1; ++j) {   // O += P V of unit j, S of unit j + 2
        const unsigned vi = (unsigned)(j - j0), ki = vi + 2, i = (unsigned)(j - first);
        const bool values = j >= j0, keys = j + 2 < j1, pv = j >= first && j < end;
        uint64_t* bv = &bars->v_full[vi % kVStages];
        uint64_t* bk = &bars->k_full[ki % kKStages];
        uint64_t* bp = &bars->p_full[x][i & 1];
        const uint32_t pv_par = (vi / kVStages) & 1, pk_par = (ki / kKStages) & 1, pp_par = (i >> 1) & 1;
        if (!(values && keys && pv && peek3(bv, pv_par, bk, pk_par, bp, pp_par))) {
          if (values) ok = ok && wait_or_abort(bv, pv_par, abort_flag);
          if (keys) ok = ok && wait_or_abort(bk, pk_par, abort_flag);
          if (pv) ok = ok && wait_or_abort(bp, pp_par, abort_flag);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int valid = n_k - first_key_of(j);
        if (values && valid < kUnit) {   // rows past the sequence may hold NaN, which a zero weight keeps: clear them
          unsigned char* vs = sm + kOffV + (vi % kVStages) * kUnitBytes;
          for (int e = lane; e < (kUnit - valid) * 16; e += 32) {
            const int r = valid + (e >> 4), c = e & 15;
            *reinterpret_cast<uint4*>(vs + (c >> 3) * kUnitBox + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc5::fence_after_sync();
        const bool scores = j + 2 >= first && j + 2 < end;
        if (elect_one()) {
          const uint32_t ti = ts + 64 * (i & 1);
          if (pv) {   // 16 keys a step: two 8-row groups of both 64-column boxes
            const uint64_t vs = dv + (vi % kVStages) * (kUnitBytes >> 4);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mma_bf16_ta(to, ti + 8 * c, vs + c * (2048 >> 4), idesc_o, j > first || c > 0);
          }
          if (scores) {
            const uint64_t ks = dk + (ki % kKStages) * (kUnitBytes >> 4);
#pragma unroll
            for (int c = 0; c < 8; ++c)
              tc5::mma_bf16(ti, dq + (((c >> 2) * kBoxBytes + (c & 3) * 32) >> 4),
                            ks + (((c >> 2) * kUnitBox + (c & 3) * 32) >> 4), idesc_s, c > 0);
          }
          // past the last unit the barrier still tells that O += P V is complete
          if (scores || pv) tc5::mma_commit(&bars->s_full[x][i & 1]);
          if (values) tc5::mma_commit(&bars->v_empty[vi % kVStages]);
          if (keys) tc5::mma_commit(&bars->k_empty[ki % kKStages]);
        }
        __syncwarp();
      }
      // every MMA done before tensor memory is freed
      __syncwarp();
      if (elect_one()) tc5::mma_commit(&bars->drain);
      mbar_wait_bounded(&bars->drain, 0, kWaitIters);
      __syncwarp();
    }
  } else {
    // softmax of block x, a thread per row = tensor-memory lane
    const int x = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = lanes + kColO + 128 * x;
    const float slope = BIAS ? p.slopes[h] * kLog2e : 0.f;
    float m = -INFINITY, l = 0.f;   // reference (log2 units) and the sum of weights
    bool ok = true;
    const int nt = t1[x] > t0[x] ? t1[x] - t0[x] : 0;
    for (int it = 0; it < nt; ++it) {
      const int base = first_key_of(t0[x] + it);
      const uint32_t ts = lanes + kColS + 128 * x + 64 * (it & 1);
      ok = wait_or_abort(&bars->s_full[x][it & 1], (it >> 1) & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc5::fence_after_sync();
      float s[kUnit];
      tmem_ld32(ts, s);
      tmem_ld32(ts + 32, s + 32);
      tc5::tmem_wait_ld();
      if (CAP) cap_scores(p, s);
      if (BIAS) {   // s qk_log2 - slope |j - i|, without the bars where no key of the unit is behind a row
        const float off = (float)(base - pos);
        const float mul = CAP ? 1.f : p.qk_log2;
        if (__all_sync(0xffffffffu, off <= (float)(1 - kUnit))) {
          const f32x2 m2 = pack2(mul, mul), sl2 = pack2(slope, slope), off2 = pack2(slope * off, slope * off);
#pragma unroll
          for (int c = 0; c < kUnit; c += 2) {
            const f32x2 bias = fma2(sl2, pack2((float)c, (float)(c + 1)), off2);
            unpack2(fma2(pack2(s[c], s[c + 1]), m2, bias), s[c], s[c + 1]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < kUnit; ++c) s[c] = fmaf(-slope, fabsf(off + (float)c), s[c] * mul);
        }
      }
      const int lo_t = lo - base, hi_t = hi - base;
      if (!__all_sync(0xffffffffu, lo_t <= 0 && hi_t >= kUnit - 1)) {
#pragma unroll
        for (int c = 0; c < kUnit; ++c)
          if (c < lo_t || c > hi_t) s[c] = -INFINITY;
      }
      float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
      for (int c = 4; c < kUnit - 4; c += 8) {
        mx0 = max3(mx0, s[c], s[c + 4]);
        mx1 = max3(mx1, s[c + 1], s[c + 5]);
        mx2 = max3(mx2, s[c + 2], s[c + 6]);
        mx3 = max3(mx3, s[c + 3], s[c + 7]);
      }
      mx0 = max3(mx0, s[kUnit - 4], s[kUnit - 3]);
      mx1 = max3(mx1, s[kUnit - 2], s[kUnit - 1]);
      constexpr bool kRaw = !CAP && !BIAS;   // s still lacks the factor qk_log2
      const float mul = kRaw ? p.qk_log2 : 1.f;
      const float mx = fmaxf(max3(mx0, mx1, mx2), mx3) * mul;
      const bool grow = mx > m + kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mx : m;
        const float f = m_new == m ? 1.f : ex2(m - m_new);   // 0 for a row's first unit
        m = m_new;
        l *= f;
        if (it > 0) {
          const int nx = it + 1;   // scores of the next unit: the last product into O is complete
          ok = __all_sync(0xffffffffu, wait_or_abort(&bars->s_full[x][nx & 1], (nx >> 1) & 1, abort_flag));
          if (!ok) break;
          tc5::fence_after_sync();
#pragma unroll 1
          for (int c = 0; c < kD; c += 32) {
            float o[32];
            tmem_ld32(to + c, o);
            tc5::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(to + c, reinterpret_cast<const uint32_t*>(o));
          }
        }
      }
      const float sub = m == -INFINITY ? 0.f : -m;
      const f32x2 mul2v = pack2(mul, mul), sub2 = pack2(sub, sub);
      f32x2 la = 0ull, lb = 0ull;
      uint32_t w[32];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        float p0, p1, p2, p3;
        unpack2(fma2(pack2(s[2 * e], s[2 * e + 1]), mul2v, sub2), p0, p1);
        unpack2(fma2(pack2(s[2 * e + 2], s[2 * e + 3]), mul2v, sub2), p2, p3);
        p0 = ex2(p0), p1 = ex2(p1), p2 = ex2(p2), p3 = ex2(p3);
        la = add2(la, pack2(p0, p1));
        lb = add2(lb, pack2(p2, p3));
        w[e] = cvt_bf16x2(p0, p1);
        w[e + 1] = cvt_bf16x2(p2, p3);
      }
      tmem_st32(ts, w);
      float l0, l1;
      unpack2(add2(la, lb), l0, l1);
      l += l0 + l1;
      tmem_wait_st();
      tc5::fence_before_sync();
      mbar_arrive(&bars->p_full[x][it & 1]);
    }
    // out = O / l; zeros for a row that saw nothing (l = 0: a row with a NaN has a NaN there)
    if (nt > 0 && ok)
      ok = __all_sync(0xffffffffu, wait_or_abort(&bars->s_full[x][(nt + 1) & 1], ((nt + 1) >> 1) & 1, abort_flag));
    if (ok && p.n_split > 1) {
      tc5::fence_after_sync();
      float* rec = p.part + ((((size_t)split * p.B + b) * p.Hq + h) * p.t_q + row) * kPart;
#pragma unroll 1
      for (int c = 0; c < kD && nt > 0; c += 32) {
        float o[32];
        tmem_ld32(to + c, o);
        tc5::tmem_wait_ld();
        if (row < n_q) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4*>(rec + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      // a row with NaN scores alone has no reference, but has seen keys: the join has to take its NaN
      if (row < n_q) rec[kD] = nt == 0 ? -INFINITY : m == -INFINITY && l != 0.f ? 0.f : m, rec[kD + 1] = l;
    } else if (ok) {
      tc5::fence_after_sync();
      const float inv = 1.f / l;
      lrkv_bf16* orow = p.out + b * p.os_b + row * p.os_t + h * p.os_h;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        float o[32];
        if (nt > 0) {
          tmem_ld32(to + c, o);
          tc5::tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (row < n_q) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = l == 0.f ? 0u : cvt_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            if (p.out32) {
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(orow + c + 2 * e),
                           "r"(w[e]), "r"(w[e + 1]), "r"(w[e + 2]), "r"(w[e + 3]), "r"(w[e + 4]),
                           "r"(w[e + 5]), "r"(w[e + 6]), "r"(w[e + 7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(orow + c + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
              *reinterpret_cast<uint4*>(orow + c + 2 * e + 8) =
                  make_uint4(w[e + 4], w[e + 5], w[e + 6], w[e + 7]);
            }
          }
        }
      }
    }
  }
  if (*abort_flag && p.dev_status && tid == 0) atomicOr(p.dev_status, LRKV_DEV_WAIT_TIMEOUT);
  tc5::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc5::fence_after_sync();
    tc5::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the splits' results: a warp per query row and head, four values to a lane.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= (long long)p.B * p.Hq * p.t_q) return;
  const int row = (int)(i % p.t_q), h = (int)(i / p.t_q % p.Hq), b = (int)(i / p.t_q / p.Hq);
  if (p.q_len && row >= p.q_len[b]) return;
  const size_t step = (size_t)p.B * p.Hq * p.t_q * kPart;
  const float* rec = p.part + (size_t)i * kPart;
  float m = -INFINITY;
  for (int s = 0; s < p.n_split; ++s) m = fmaxf(m, rec[s * step + kD]);
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < p.n_split; ++s) {
    const float* r = rec + s * step;
    if (r[kD] == -INFINITY) continue;   // nothing was seen: its values were not written
    const float w = ex2(r[kD] - m);
    const float4 v = *reinterpret_cast<const float4*>(r + 4 * lane);
    l = fmaf(w, r[kD + 1], l);
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
  }
  const float inv = 1.f / l;
  *reinterpret_cast<uint2*>(p.out + b * p.os_b + row * p.os_t + h * p.os_h + 4 * lane) =
      l == 0.f ? make_uint2(0u, 0u) : make_uint2(cvt_bf16x2(o.x * inv, o.y * inv), cvt_bf16x2(o.z * inv, o.w * inv));
}

}  // namespace prefill
}  // namespace lrkv
