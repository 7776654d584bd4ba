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
// block, not only of the other one.  
//
// Bound: a unit of both blocks costs 2 x 2 x 2 x 128 x 64 x 128 tensor flops and
// 2 x 128 x 64 exponentials; at 8192 flops and 16 exponentials a clock and SM both take
// 1024 clocks (1148 measured for the products: S with N = 64 reads shared memory at
// 48 clocks per step where 32 would do).  The groups compute their exponentials in
// turn, 770 clocks a unit each, beside the other group's loads, maxima and stores: a
// unit of both blocks takes 1555 clocks, and a CTA 11000 more before its first and after
// its last one.  8192 causal tokens x 32 heads: 473 us (1161 TFLOP/s at 1.66 GHz, the
// power limit's clock); with tiles of 128 keys, whose S has to wait for O += P V of the
// tile before, 511 us; with one MMA warp for both blocks, whose waits at four barriers a
// unit took 1200 clocks, 689 us; without the turns 485 us.
//
// The running reference m only moves when a row's maximum passes it by more than
// 2^8 (weights then stay below 2^8, and the row's sum is in fp32): O is rescaled
// in tensor memory a few times per row instead of once per unit.  The group that does
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
constexpr float kLazy = 8.f;                // rescale when a maximum grows by more (log2)

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
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2][2], p_full[2][2];   // [block][unit & 1]
  uint64_t tail_full;                    // values of a last unit that ends inside it, before they are cleared
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int lo[2], hi[2];    // union of the rows' key intervals, per block
};
static_assert(sizeof(Bars) <= 256, "barrier region");

// s[c] = softcap log2(e) tanh(scale s[c] / softcap).  Where all |x| = |scale s / softcap| of
// the warp are at most 1, as sane logits are, by a polynomial in x^2 on the two-wide fp32
// pipe (a least-squares fit of tanh(x) / x, weighted towards equal relative errors: 6.5e-7
// at most with fp32 rounding, 4e-5 in the exponent at softcap 50); else by
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

// Weights 2^(s mul + sub) of a row's unit as packed bf16, and the two halves of their sum
// before rounding.  (A quarter or half of them by a cubic polynomial on the fp32 pipe, which
// has 10 clocks of work for what the special-function unit does in 8: no faster.)
__device__ __forceinline__ f32x2 weights(const float (&s)[kUnit], float mul, float sub, uint32_t (&w)[32]) {
  const f32x2 m2 = pack2(mul, mul), sub2 = pack2(sub, sub);
  f32x2 sum[2] = {0ull, 0ull};
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    float p0, p1;
    unpack2(fma2(pack2(s[2 * e], s[2 * e + 1]), m2, sub2), p0, p1);
    p0 = ex2(p0), p1 = ex2(p1);
    sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
    w[e] = cvt_bf16x2(p0, p1);
  }
  return add2(sum[0], sum[1]);
}

template <bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(sm + kOffBar);
  volatile int* abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  // the last query blocks first: under a causal mask they are the longest
  const int hb = blockIdx.x % (p.Hq * p.B);
  const int h = hb % p.Hq, b = hb / p.Hq;
  const int blk = p.n_blocks - 1 - blockIdx.x / (p.Hq * p.B);
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
  if (bad && p.dev_status && tid == 0 && blk == 0 && h == 0) atomicOr(p.dev_status, bad);
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
    mbar_init(&bars->tail_full, 1);
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
  const int j0 = min(t0[0], t0[1]), j1 = max(t1[0], t1[1]);

  if (warp == kTmaWarp) {
    const int tail = n_k / kUnit;   // the unit that the sequence ends inside of
    const bool clear = n_k % kUnit != 0 && tail >= j0 && tail < j1;
    unsigned char* tail_v = sm + kOffV + (unsigned)(tail - j0) % kVStages * kUnitBytes;
    bool ok = true;
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
      auto load = [&](const CUtensorMap* map, uint64_t* full, uint64_t* empty, int off, int ns, int j, uint64_t* bar) {
        const int i = j - j0, s = i % ns;
        if (i >= ns && !wait_or_abort(&empty[s], ((i / ns) - 1) & 1, abort_flag)) return false;
        if (!bar) bar = &full[s];
        mbar_arrive_expect_tx(bar, kUnitBytes);
        unsigned char* dst = sm + off + s * kUnitBytes;
        tma_load_4d(dst, map, 0, hk, j * kUnit, b, bar);
        tma_load_4d(dst + kUnitBox, map, 64, hk, j * kUnit, b, bar);
        return true;
      };
      int nk = 0, nv = 0;   // units loaded
      for (int j = j0 - 2; ok && j < j1; ++j) {
        if (j + 2 < j1) {
          ok = load(&p.map_k, bars->k_full, bars->k_empty, kOffK, kKStages, j + 2, nullptr);
          if (!ok) break;
          ++nk;
        }
        if (j < j0) continue;
        const bool last = clear && j == tail;   // the last unit of all, if it is one of them
        ok = load(&p.map_v, bars->v_full, bars->v_empty, kOffV, kVStages, j, last ? &bars->tail_full : nullptr);
        if (ok && !last) ++nv;
        if (ok && last) ok = wait_or_abort(&bars->tail_full, 0, abort_flag);
      }
      // leave no copy in flight: wait for the last fill of every stage
      mbar_wait_bounded(&bars->q_full, 0, kWaitIters);
      for (int i = nk > kKStages ? nk - kKStages : 0; i < nk; ++i)
        mbar_wait_bounded(&bars->k_full[i % kKStages], (i / kKStages) & 1, kWaitIters);
      for (int i = nv > kVStages ? nv - kVStages : 0; i < nv; ++i)
        mbar_wait_bounded(&bars->v_full[i % kVStages], (i / kVStages) & 1, kWaitIters);
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (ok && clear) {   // rows past the sequence may hold NaN, which a zero weight keeps: clear them
      const int valid = n_k % kUnit;
      for (int e = lane; e < (kUnit - valid) * 16; e += 32) {
        const int r = valid + (e >> 4), c = e & 15;
        *reinterpret_cast<uint4*>(tail_v + (c >> 3) * kUnitBox + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->v_full[(unsigned)(tail - j0) % kVStages]);
    }
  } else if (warp >= kMmaWarp) {
    if (j0 < j1 && elect_one()) {   // one thread does it all
      const int x = warp - kMmaWarp, first = x ? t0[1] : t0[0], end = x ? t1[1] : t1[0];
      constexpr uint32_t idesc_s = tc5::idesc_bf16_f32(kTile, kUnit);
      constexpr uint32_t idesc_o = idesc_bf16_f32_bt(kTile, kD);
      const uint32_t ts = tmem + kColS + 128 * x, to = tmem + kColO + 128 * x;
      // descriptors of the first operands; an offset in shared memory adds its sixteenths
      const uint64_t dq = tc5::smem_desc(smem_u32(sm + kOffQ + x * kTileBytes), 16, 1024, tc5::kSwizzle128B);
      const uint64_t dk = tc5::smem_desc(smem_u32(sm + kOffK), 16, 1024, tc5::kSwizzle128B);
      const uint64_t dv = tc5::smem_desc(smem_u32(sm + kOffV), kUnitBox, 1024, tc5::kSwizzle128B);
      bool ok = wait_or_abort(&bars->q_full, 0, abort_flag);
      // A look at a barrier takes 90 clocks, beside busy warps up to 300: a step's values and keys are
      // waited for before its P can be there, so that only the wait for P stands in its way.
      auto ready = [&](int j) {
        const unsigned vi = (unsigned)(j - j0), ki = vi + 2;
        if (j + 2 < j1) ok = ok && wait_or_abort(&bars->k_full[ki % kKStages], (ki / kKStages) & 1, abort_flag);
        if (j >= j0 && j < j1) ok = ok && wait_or_abort(&bars->v_full[vi % kVStages], (vi / kVStages) & 1, abort_flag);
      };
      ready(j0 - 2);
      for (int j = j0 - 2; j < j1; ++j) {   // O += P V of unit j, S of unit j + 2
        const unsigned vi = (unsigned)(j - j0), ki = vi + 2, i = (unsigned)(j - first);
        const bool values = j >= j0, keys = j + 2 < j1, pv = j >= first && j < end;
        if (pv) ok = ok && wait_or_abort(&bars->p_full[x][i & 1], (i >> 1) & 1, abort_flag);
        if (!ok) break;
        tc5::fence_after_sync();
        const bool scores = j + 2 >= first && j + 2 < end;
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
          for (int c = 0; c < 8; ++c) {
            tc5::mma_bf16(ti, dq + (((c >> 2) * kBoxBytes + (c & 3) * 32) >> 4),
                          ks + (((c >> 2) * kUnitBox + (c & 3) * 32) >> 4), idesc_s, c > 0);
          }
        }
        // past the last unit the barrier still tells that O += P V is complete
        if (scores || pv) tc5::mma_commit(&bars->s_full[x][i & 1]);
        if (values) tc5::mma_commit(&bars->v_empty[vi % kVStages]);
        if (keys) tc5::mma_commit(&bars->k_empty[ki % kKStages]);
        ready(j + 1);
      }
      // every MMA done before tensor memory is freed
      tc5::mma_commit(&bars->drain);
      mbar_wait_bounded(&bars->drain, 0, kWaitIters);
    }
    __syncwarp();
  } else {
    // softmax of block x, a thread per row = tensor-memory lane
    const int x = warp >> 2;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = lanes + kColO + 128 * x;
    const float slope = BIAS ? p.slopes[h] * kLog2e : 0.f;
    float m = -INFINITY, l = 0.f;   // reference (log2 units) and the sum of weights
    bool ok = true;
    const int nt = t1[x] - t0[x];
    // The groups compute exponentials in turn (named barriers 1 and 2), unit by unit of both
    // blocks: what else a unit takes runs beside the other group's exponentials.
    auto my_turn = [&]() { tc5::named_bar_sync(1 + x, 2 * kTile); };
    auto your_turn = [&](int j) {
      if (x == 0 || j + 1 < j1) tc5::named_bar_arrive(2 - x, 2 * kTile);
    };
    if (x == 1 && j0 < j1) tc5::named_bar_arrive(1, 2 * kTile);
    bool seen = false;   // this unit's scores are known to be there
    for (int j = j0; j < j1; ++j) {
      const int it = j - t0[x], base = j * kUnit;
      const uint32_t ts = lanes + kColS + 128 * x + 64 * (it & 1);
      const bool here = it >= 0 && it < nt;
      if (here && !seen) ok = __all_sync(0xffffffffu, ok && wait_or_abort(&bars->s_full[x][it & 1], (it >> 1) & 1, abort_flag));
      if (!here || !ok) {   // both groups take every turn
        my_turn();
        your_turn(j);
        continue;
      }
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
      const bool whole = __all_sync(0xffffffffu, lo_t <= 0 && hi_t >= kUnit - 1);
      if (!whole) {
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
          tc5::fence_after_sync();
#pragma unroll 1
          for (int c = 0; ok && c < kD; c += 32) {
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
      uint32_t w[32];
      my_turn();
      const f32x2 sum = weights(s, mul, sub, w);
      your_turn(j);
      // the next unit's scores are mostly there by now: the look at their barrier overlaps the stores
      seen = __all_sync(0xffffffffu, mbar_test(&bars->s_full[x][(it + 1) & 1], ((it + 1) >> 1) & 1));
      tmem_st32(ts, w);
      float l0, l1;
      unpack2(sum, l0, l1);
      l += l0 + l1;
      tmem_wait_st();
      tc5::fence_before_sync();
      mbar_arrive(&bars->p_full[x][it & 1]);
    }
    // out = O / l; zeros for a row that saw nothing
    if (nt > 0 && ok)
      ok = __all_sync(0xffffffffu, wait_or_abort(&bars->s_full[x][(nt + 1) & 1], ((nt + 1) >> 1) & 1, abort_flag));
    if (ok) {
      tc5::fence_after_sync();
      const float inv = l > 0.f ? 1.f / l : 0.f;
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
            w[e] = l > 0.f ? cvt_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
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

}  // namespace prefill
}  // namespace lrkv
