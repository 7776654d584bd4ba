// What the kernels of the paged 8-bit cache share: sizes, the workspace, and the
// conversions between 8-bit codes and wider types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../lrkv_common.cuh"
#include "../ptx.cuh"
#include "lrkv_serve.h"
#include "serve_host.cuh"
#include "serve_ptx.cuh"

namespace lrkv {
namespace paged {

using namespace serve;

constexpr float kTinyScale = 7.888609052210118e-31f;   // 2^-100

// Codes of one page of one layer (keys or values).
__host__ __device__ __forceinline__ size_t page_elems(const lrkv_paged_dims& D) {
  return (size_t)D.Hkv * D.page * kD;
}

// e4m3 codes: two floats to two codes (nearest even, finite), `lo` in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two e4m3 codes (16 bits) to f16x2, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  return d;
}
// Four codes of a word as f16x2 of bytes (0, 1) and of bytes (2, 3), exactly.
template <int CODE>
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& h01, uint32_t& h23) {
  if (CODE == LRKV_CODE_INT8) {
    s8x4_f16pairs(w, h01, h23);
  } else {
    h01 = e4m3x2_f16x2(w & 0xffffu);
    h23 = e4m3x2_f16x2(w >> 16);
  }
}
__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Four codes of a word as fp32, exactly.
template <int CODE>
__device__ __forceinline__ void codes_f32(uint32_t w, float (&x)[4]) {
  uint32_t a, b;
  codes_f16<CODE>(w, a, b);
  const float2 u = f16x2_f32(a), v = f16x2_f32(b);
  x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
}
// Four values in units of the scale (|t| <= Q (1 + 2^-22)) to four codes, nearest
// even.  int8: t + 1.5 2^23 holds the nearest integer of t in its low byte, two's
// complement (the rounding of the sum, in fp32, is the rounding to an integer; t
// has been rounded before, so the sum must not be fused with t's product).
template <int CODE>
__device__ __forceinline__ uint32_t pack_codes(float t0, float t1, float t2, float t3) {
  if (CODE == LRKV_CODE_INT8) {
    const uint32_t r0 = __float_as_uint(__fadd_rn(t0, 12582912.f)), r1 = __float_as_uint(__fadd_rn(t1, 12582912.f));
    const uint32_t r2 = __float_as_uint(__fadd_rn(t2, 12582912.f)), r3 = __float_as_uint(__fadd_rn(t3, 12582912.f));
    return __byte_perm(__byte_perm(r0, r1, 0x0040), __byte_perm(r2, r3, 0x0040), 0x5410);
  }
  return cvt_e4m3x2(t0, t1) | (cvt_e4m3x2(t2, t3) << 16);
}

inline lrkv_status check_dims(const lrkv_paged_dims* D) {
  if (!D) return LRKV_ERR_INVALID_ARG;
  if (D->B < 1 || D->Hq < 1 || D->Hkv < 1 || D->n_pages < 1 || D->max_pages < 1 || D->n_layers < 1)
    return LRKV_ERR_INVALID_ARG;
  if (D->Hq % D->Hkv) return LRKV_ERR_INVALID_ARG;
  if (D->code != LRKV_CODE_INT8 && D->code != LRKV_CODE_E4M3) return LRKV_ERR_INVALID_ARG;
  if (D->page != 16 && D->page != 32 && D->page != 64 && D->page != 128) return LRKV_ERR_INVALID_ARG;
  if (D->d != kD || D->B > 65535 || D->Hkv > 65535 || D->Hq / D->Hkv > kMaxG) return LRKV_ERR_UNSUPPORTED;
  // positions are 32-bit, and exact in fp32 for the distance bias
  if ((long long)D->max_pages * D->page > (1LL << 24)) return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

inline lrkv_status check_cache(const lrkv_paged_cache* C) {
  if (!C) return LRKV_ERR_INVALID_ARG;
  const void* ptrs[] = {C->k, C->v, C->scale_k, C->scale_v, C->page_table, C->seq_len, C->refs, C->dev_status};
  for (const void* p : ptrs)
    if (!p) return LRKV_ERR_INVALID_ARG;
  for (const void* p : ptrs)
    if (!aligned16(p)) return LRKV_ERR_ALIGNMENT;
  return LRKV_OK;
}

inline lrkv_status check_all(const lrkv_paged_dims* D, const lrkv_paged_cache* C) {
  const lrkv_status st = check_dims(D);
  return st != LRKV_OK ? st : check_cache(C);
}

// Tokens of sequence b in this call: t_new, or t_new_b[b] clamped into [0, t_new].
__device__ __forceinline__ int call_tokens(const int32_t* t_new_b, int b, int t_new, uint32_t* status) {
  uint32_t st = 0;
  const int n = new_tokens(t_new_b, b, t_new, &st);
  *status |= st;
  return n;
}

// The workspace of the paged calls, offsets in bytes.  Everything that has to be
// zero between calls lies in front.
constexpr int kMaxTq = 64;             // query tokens per sequence of lrkv_paged_attn
constexpr int kMaxRowBlocks = 4;      // 8-row blocks that a CTA of lrkv_paged_attn holds
// A row's partial result: values (rows 136 floats apart, so that the 4 rows of a quad of
// lanes lie in different banks), reference, sum.
constexpr int kRecRow = kD + 8, kRecFloats = kRecRow + 2;
// Warps of a lrkv_paged_attn CTA that holds nb blocks of 8 query rows: as many as their
// accumulators leave registers for.
__host__ __device__ constexpr int attn_warps(int nb) { return nb == 1 ? 16 : 8; }
struct PagedWs {
  size_t tickets;   // int32 [ctas]: arrivals at a sequence that several CTAs share; zero between calls
  size_t claims;    // int32 [max(n_pages, B)]: who named an index first; zero between calls
  size_t ticket;    // int32 [4]: arrivals of a list call's CTAs; zero between calls
  size_t list;      // int32 [4 + 5 max(n_pages, B)]: counts, then lists of pages
  size_t recs;      // float [ctas][2 + warps][rows][kRecFloats]
  size_t total;
  int ctas, rows, row_blocks;   // rows: padded rows per row block
};

// Rows of one kv head (g t_q) in blocks, evenly, each padded to 8.  A block reads the cache
// once: of up to 32 rows where a layer's page tables have room for more than L2 holds (100 tiles
// of 32 tokens for every SM, 121 MB), of up to 8 where they do not, as the kernel for 8 rows has
// twice the warps and less to fetch and join.  (The lengths lie on the device: a table with
// room for a long context takes the large blocks while its sequences are short, too.)  Measured with 20 rows: 7 sequences of 2500 to 5000 tokens 50 us in
// blocks of 8, 58 us in one; of 20000 to 40000 tokens 209 and 166 us.
inline PagedWs paged_ws(const lrkv_paged_dims& D, int t_q) {
  PagedWs L;
  L.ctas = num_sms();
  const int rows = D.Hq / D.Hkv * t_q;
  const long long tiles = (long long)D.B * D.Hkv * (((long long)D.max_pages * D.page + 31) / 32);
  const int most = tiles <= 100LL * L.ctas ? 8 : 8 * kMaxRowBlocks;
  L.row_blocks = (rows + most - 1) / most;
  L.rows = ((rows + L.row_blocks - 1) / L.row_blocks + 7) / 8 * 8;
  const size_t n = (size_t)(D.n_pages > D.B ? D.n_pages : D.B);
  size_t off = 0;
  L.ticket = off;
  off = align_up(off + 4 * sizeof(int32_t), 256);
  L.claims = off;
  off = align_up(off + n * sizeof(int32_t), 256);
  L.tickets = off;
  off = align_up(off + L.ctas * sizeof(int32_t), 256);
  L.list = off;
  off = align_up(off + (4 + 5 * n) * sizeof(int32_t), 256);
  L.recs = off;
  off = align_up(off + sizeof(float) * L.ctas * (2 + attn_warps(L.rows / 8)) * (size_t)L.rows * kRecFloats, 256);
  L.total = off;
  return L;
}

}  // namespace paged
}  // namespace lrkv
