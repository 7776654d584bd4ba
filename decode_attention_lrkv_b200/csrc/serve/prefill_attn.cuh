// Prefill attention on the 5th-generation tensor cores.
//
// For every query row i of a head:  o_i = sum_j p_ij v_j / sum_j p_ij,
// p_ij = exp(s_ij - m_i), s_ij the modified scores (lrkv_score), m_i a running
// reference close to the row's maximum; one pass over the keys in tiles of 128.
//
// A CTA takes two blocks of 128 query rows (X = 0, 1) of one head.  Per key tile
// and block:
//     S_X = Q_X K^T      (M 128, N 128, K 128; operands in shared memory)
//     P_X = exp2(S_X ..) (a thread per row; P_X overwrites S_X as packed bf16)
//     O_X += P_X V       (M 128, N 128, K 128; P_X read from tensor memory)
// S_0, S_1, O_0, O_1 fill the 512 columns of tensor memory.  One warp issues TMA
// loads (128-byte swizzle, rings of key and value tiles), one issues MMAs, two
// groups of four warps do the softmax of a block each.  The MMA warp alternates
// between the blocks, so the tensor cores work on one block while the other's
// softmax runs.
//
// Bound: a tile pair costs 2 x 2 x 2 x 128^3 tensor flops and 2 x 128^2
// exponentials; at 8192 flops and 16 exponentials a clock and SM both take 2048
// clocks, so the softmax's instruction count decides.
//
// The running reference m only moves when a row's maximum passes it by more than
// 2^8 (weights then stay below 2^8, and the row's sum is in fp32): O is rescaled
// in tensor memory a few times per row instead of once per tile.  A softmax group
// may touch O_X right after it sees S_X complete: MMAs complete in order, and the
// next product into O_X waits for this group's P_X.
//
// Every mask is an interval [lo, hi] of keys per row, so a block's tiles are the
// union of its rows' intervals, and a tile inside all of a warp's intervals is not
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

constexpr int kTile = 128;                  // query rows per block, keys per tile
constexpr int kThreads = 320;               // warps 0-3, 4-7 softmax of block 0, 1; 8 TMA; 9 MMA
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kTileBytes = kTile * kD * 2;  // two boxes of 64 columns
constexpr int kBoxBytes = kTileBytes / 2;
constexpr int kKStages = 2, kVStages = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 X
constexpr float kLazy = 8.f;                // rescale when a maximum grows by more (log2)

// Shared memory: Q blocks, key ring, value ring (each 1024-aligned), barriers.
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kTileBytes;
constexpr int kOffV = kOffK + kKStages * kTileBytes;
constexpr int kOffBar = kOffV + kVStages * kTileBytes;
constexpr size_t kSmemBytes = kOffBar + 256 + 1024;

struct Params {
  CUtensorMap map_q, map_k, map_v;   // [B][t][H][128] as (128, H, t, B), box {64, 1, 128, 1}
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
  float cap_in;       // 2 log2(e) scale / softcap
  float cap_log2;     // softcap * log2(e)
  int out32;          // 32-byte stores allowed
};

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int lo[2], hi[2];    // union of the rows' key intervals, per block
};
static_assert(sizeof(Bars) <= 256, "barrier region");

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
    for (int s = 0; s < kKStages; ++s) mbar_init(&bars->k_full[s], 1), mbar_init(&bars->k_empty[s], 1);
    for (int s = 0; s < kVStages; ++s) mbar_init(&bars->v_full[s], 1), mbar_init(&bars->v_empty[s], 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars->s_full[x], 1);
      mbar_init(&bars->p_full[x], kTile);
      mbar_init(&bars->o_full[x], 1);
      bars->lo[x] = 0x7fffffff;
      bars->hi[x] = -1;
    }
    mbar_init(&bars->drain, 1);
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
  // tiles [t0[x], t1[x]) of block x; [j0, j1) of the CTA
  int t0[2], t1[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const bool any = bars->hi[x] >= 0;
    t0[x] = __shfl_sync(0xffffffffu, any ? bars->lo[x] / kTile : 0x7fffffff, 0);   // known to be uniform
    t1[x] = __shfl_sync(0xffffffffu, any ? bars->hi[x] / kTile + 1 : 0, 0);
  }
  const int j0 = min(t0[0], t0[1]), j1 = max(t1[0], t1[1]);

  if (warp == kTmaWarp) {
    if (lane == 0 && j0 < j1) {
      mbar_arrive_expect_tx(&bars->q_full, 2 * kTileBytes);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tma_load_4d(sm + kOffQ + x * kTileBytes + c * kBoxBytes, &p.map_q, 64 * c, h, row0 + x * kTile, b,
                      &bars->q_full);
      auto load = [&](const CUtensorMap* map, uint64_t* full, uint64_t* empty, int off, int ns, int j) {
        const int i = j - j0, s = i % ns;
        if (i >= ns && !wait_or_abort(&empty[s], ((i / ns) - 1) & 1, abort_flag)) return false;
        mbar_arrive_expect_tx(&full[s], kTileBytes);
        unsigned char* dst = sm + off + s * kTileBytes;
        tma_load_4d(dst, map, 0, hk, j * kTile, b, &full[s]);
        tma_load_4d(dst + kBoxBytes, map, 64, hk, j * kTile, b, &full[s]);
        return true;
      };
      int nk = 0, nv = 0;   // tiles loaded
      bool ok = load(&p.map_k, bars->k_full, bars->k_empty, kOffK, kKStages, j0);
      if (ok) ++nk;
      for (int j = j0; ok && j < j1; ++j) {
        if (j + 1 < j1) {
          ok = load(&p.map_k, bars->k_full, bars->k_empty, kOffK, kKStages, j + 1);
          if (!ok) break;
          ++nk;
        }
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
  } else if (warp == kMmaWarp) {
    if (j0 < j1) {
      constexpr uint32_t idesc_s = tc5::idesc_bf16_f32(kTile, kTile);
      constexpr uint32_t idesc_o = idesc_bf16_f32_bt(kTile, kD);
      // descriptors of the first operands; an offset in shared memory adds its sixteenths
      const uint64_t dq = tc5::smem_desc(smem_u32(sm + kOffQ), 16, 1024, tc5::kSwizzle128B);
      const uint64_t dk = tc5::smem_desc(smem_u32(sm + kOffK), 16, 1024, tc5::kSwizzle128B);
      const uint64_t dv = tc5::smem_desc(smem_u32(sm + kOffV), kBoxBytes, 1024, tc5::kSwizzle128B);
      auto issue_s = [&](int x, int j) {   // S_x = Q_x K_j^T
        if (elect_one()) {
          const uint64_t ks = dk + ((j - j0) % kKStages) * (kTileBytes >> 4), qs = dq + x * (kTileBytes >> 4);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint32_t off = ((c >> 2) * kBoxBytes + (c & 3) * 32) >> 4;
            tc5::mma_bf16(tmem + kColS + 128 * x, qs + off, ks + off, idesc_s, c > 0);
          }
          tc5::mma_commit(&bars->s_full[x]);
        }
      };
      auto issue_o = [&](int x, int j) {   // O_x += P_x V_j
        if (elect_one()) {
          const uint64_t vs = dv + ((j - j0) % kVStages) * (kTileBytes >> 4);
#pragma unroll
          for (int c = 0; c < 8; ++c)      // 16 keys: two 8-row groups of both 64-column boxes
            mma_bf16_ta(tmem + kColO + 128 * x, tmem + kColS + 128 * x + 8 * c, vs + c * (2048 >> 4), idesc_o,
                        j > t0[x] || c > 0);
          if (j == t1[x] - 1) tc5::mma_commit(&bars->o_full[x]);
        }
      };
      bool ok = wait_or_abort(&bars->q_full, 0, abort_flag) && wait_or_abort(&bars->k_full[0], 0, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc5::fence_after_sync();
        for (int x = 0; x < 2; ++x)
          if (t0[x] == j0) issue_s(x, j0);
        if (elect_one()) tc5::mma_commit(&bars->k_empty[0]);
      }
      int done[2] = {0, 0};   // P tiles taken per block
      for (int j = j0; ok && j < j1; ++j) {
        const int vi = j - j0, ki = vi + 1;
        const bool more = j + 1 < j1;
        ok = wait_or_abort(&bars->v_full[vi % kVStages], (vi / kVStages) & 1, abort_flag);
        if (ok && more) ok = wait_or_abort(&bars->k_full[ki % kKStages], (ki / kKStages) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int valid = n_k - j * kTile;
        if (valid < kTile) {   // rows past the sequence may hold NaN, which a zero weight keeps: clear them
          unsigned char* vs = sm + kOffV + (vi % kVStages) * kTileBytes;
          for (int e = lane; e < (kTile - valid) * 16; e += 32) {
            const int r = valid + (e >> 4), c = e & 15;
            *reinterpret_cast<uint4*>(vs + (c >> 3) * kBoxBytes + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (j >= t0[x] && j < t1[x]) {
            ok = ok && wait_or_abort(&bars->p_full[x], done[x] & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++done[x];
            tc5::fence_after_sync();
            issue_o(x, j);
          }
          if (more && j + 1 >= t0[x] && j + 1 < t1[x]) issue_s(x, j + 1);
        }
        if (!ok) break;
        if (elect_one()) {
          tc5::mma_commit(&bars->v_empty[vi % kVStages]);
          if (more) tc5::mma_commit(&bars->k_empty[ki % kKStages]);
        }
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
    const uint32_t ts = lanes + kColS + 128 * x, to = lanes + kColO + 128 * x;
    const float slope = BIAS ? p.slopes[h] * kLog2e : 0.f;
    float m = -INFINITY, l = 0.f;   // reference (log2 units) and the sum of weights
    bool ok = true;
    const int nt = t1[x] - t0[x];
    for (int it = 0; it < nt; ++it) {
      const int base = (t0[x] + it) * kTile;
      ok = wait_or_abort(&bars->s_full[x], it & 1, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc5::fence_after_sync();
      float s[kTile];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s + 32 * c);
      tc5::tmem_wait_ld();
      if (CAP) {   // softcap tanh(s / softcap) = softcap (1 - 2 / (1 + e^(2 s / softcap)))
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          s[c] = fmaf(-2.f * p.cap_log2, rcp_fast(1.f + ex2(s[c] * p.cap_in)), p.cap_log2);
      }
      if (BIAS) {
        const float off = (float)(base - pos);
#pragma unroll
        for (int c = 0; c < kTile; ++c) {
          const float v = CAP ? s[c] : s[c] * p.qk_log2;
          s[c] = fmaf(-slope, fabsf(off + (float)c), v);
        }
      }
      const int lo_t = lo - base, hi_t = hi - base;
      if (!__all_sync(0xffffffffu, lo_t <= 0 && hi_t >= kTile - 1)) {
#pragma unroll
        for (int c = 0; c < kTile; ++c)
          if (c < lo_t || c > hi_t) s[c] = -INFINITY;
      }
      float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
      for (int c = 4; c < kTile; c += 4) {
        mx0 = fmaxf(mx0, s[c]);
        mx1 = fmaxf(mx1, s[c + 1]);
        mx2 = fmaxf(mx2, s[c + 2]);
        mx3 = fmaxf(mx3, s[c + 3]);
      }
      constexpr bool kRaw = !CAP && !BIAS;   // s still lacks the factor qk_log2
      const float mul = kRaw ? p.qk_log2 : 1.f;
      const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * mul;
      const bool grow = mx > m + kLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? mx : m;
        const float f = m_new == m ? 1.f : ex2(m - m_new);   // 0 for a row's first tile
        m = m_new;
        l *= f;
        if (it > 0) {
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
      float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
      for (int c = 0; c < kTile; c += 64) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float p0 = ex2(fmaf(s[c + 2 * e], mul, sub)), p1 = ex2(fmaf(s[c + 2 * e + 1], mul, sub));
          const float p2 = ex2(fmaf(s[c + 2 * e + 2], mul, sub)), p3 = ex2(fmaf(s[c + 2 * e + 3], mul, sub));
          l0 += p0, l1 += p1, l2 += p2, l3 += p3;
          w[e] = cvt_bf16x2(p0, p1);
          w[e + 1] = cvt_bf16x2(p2, p3);
        }
        tmem_st32(ts + c / 2, w);
      }
      l += (l0 + l1) + (l2 + l3);
      tmem_wait_st();
      tc5::fence_before_sync();
      mbar_arrive(&bars->p_full[x]);
    }
    // out = O / l; zeros for a row that saw nothing
    if (nt > 0 && ok) ok = __all_sync(0xffffffffu, wait_or_abort(&bars->o_full[x], 0, abort_flag));
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
