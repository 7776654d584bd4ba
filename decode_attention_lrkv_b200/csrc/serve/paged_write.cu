// lrkv_paged_append and lrkv_paged_read: bf16 rows into the 8-bit pages, one scale
// per page and head, and back.
//
// Append: a CTA per (page that the call touches, kv head, sequence); threads 0-127
// take the keys, 128-255 the values.  Every thread holds its part of the page's new
// rows in registers (16 elements per row piece, page / 16 pieces), so the rows are
// read once: load, maximum over the page (a packed 16-bit maximum of the bf16
// magnitudes, whose bit patterns are ordered), scale, codes, 16-byte stores.  Where
// a page held tokens before and its scale has grown, their codes are rounded again
// in place.  Bound by memory: 2 d bytes in and d out per row.
//
// Read: eight threads per row, 16 codes in and 32 bytes out each; keys and values of
// a row by the same threads, two rows in flight.  Bound by memory: d in, 2 d out.  32768
// tokens x 32 heads: append 123 us, read 125 us (6.5 TB/s each); read with two 16-byte stores
// in place of one of 32 bytes 141 us, with one or four rows in flight 125.
#include "paged.cuh"

#include "../launch_util.cuh"

namespace lrkv {
namespace paged {

struct AppendParams {
  lrkv_paged_dims D;
  lrkv_paged_cache C;
  const lrkv_bf16* k_new;
  const lrkv_bf16* v_new;
  const int32_t* t_new_b;
  int layer, t_new, touched;   // pages that a sequence's tokens can touch
};

constexpr int kAppendThreads = 256;

// Non-finite bf16 magnitudes of a pair: NaN to 0, infinity to the largest finite.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t x = (w >> (16 * i)) & 0xffffu;
    const uint32_t mag = x & 0x7fffu;
    if (mag > 0x7f80u) x = 0;
    else if (mag == 0x7f80u) x = (x & 0x8000u) | 0x7f7fu;
    r |= x << (16 * i);
  }
  return r;
}

template <int PAGE, int CODE>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kPieces = PAGE / 16;   // 16-element pieces per thread
  constexpr float Q = CODE == LRKV_CODE_INT8 ? 127.f : 448.f;
  __shared__ uint32_t s_max[2][4];
  griddep_wait();
  griddep_launch_dependents();
  const lrkv_paged_dims& D = p.D;
  const int h = blockIdx.x % D.Hkv, w = blockIdx.x / D.Hkv, b = blockIdx.y;
  const int side = threadIdx.x >> 7, t = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  uint32_t status = 0;
  const int n = call_tokens(p.t_new_b, b, p.t_new, &status);
  const int cap = D.max_pages * PAGE;
  const int start = min(max(p.C.seq_len[b], 0), cap);
  int stop = start + n;
  if (stop > cap) status |= LRKV_DEV_SEQ_OVERFLOW, stop = cap;
  if (status && h == 0 && w == 0 && threadIdx.x == 0) atomicOr(p.C.dev_status, status);
  const int slot = start / PAGE + w, first = slot * PAGE;   // this page's first position
  if (first >= stop || n == 0) return;
  const int r0 = max(start - first, 0), r1 = min(stop - first, PAGE);   // rows of this call
  const int pid = p.C.page_table[(size_t)b * D.max_pages + slot];
  if (pid < 0 || pid >= D.n_pages) {
    if (threadIdx.x == 0) atomicOr(p.C.dev_status, LRKV_DEV_BAD_PAGE);
    return;
  }
  const size_t ph = ((size_t)p.layer * D.n_pages + pid) * D.Hkv + h;
  unsigned char* codes = static_cast<unsigned char*>(side == 0 ? p.C.k : p.C.v) + ph * PAGE * kD;
  float* scale = (side == 0 ? p.C.scale_k : p.C.scale_v) + ph;
  const lrkv_bf16* src = (side == 0 ? p.k_new : p.v_new) +
                         (((ptrdiff_t)b * p.t_new + (first - start)) * D.Hkv + h) * kD;   // row 0 of the page
  uint32_t x[kPieces][8];
  uint32_t mx = 0;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int r = (t >> 3) + 16 * k, c = (t & 7) * 16;
    uint4 a = make_uint4(0, 0, 0, 0), e = a;
    if (r >= r0 && r < r1) {
      const uint4* g = reinterpret_cast<const uint4*>(src + (ptrdiff_t)r * D.Hkv * kD + c);
      a = __ldcs(g);
      e = __ldcs(g + 1);
    }
    x[k][0] = a.x, x[k][1] = a.y, x[k][2] = a.z, x[k][3] = a.w;
    x[k][4] = e.x, x[k][5] = e.y, x[k][6] = e.z, x[k][7] = e.w;
  }
  const float before = r0 > 0 ? *scale : 0.f;
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = __vmaxu2(mx, x[k][i] & 0x7fff7fffu);
  if ((mx & 0xffffu) >= 0x7f80u || (mx >> 16) >= 0x7f80u) {   // infinities or NaN: rare
    mx = 0;
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[k][i] = finite_pair(x[k][i]);
        mx = __vmaxu2(mx, x[k][i] & 0x7fff7fffu);
      }
  }
  mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
  if ((t & 31) == 0) s_max[side][warp] = mx;
  __syncthreads();
  mx = max(max(s_max[side][0], s_max[side][1]), max(s_max[side][2], s_max[side][3]));
  float s = fmaxf(before, __fdiv_rn(__uint_as_float(mx << 16), Q));
  if (s < kTinyScale) s = 0.f;
  const float inv = s > 0.f ? __fdiv_rn(1.f, s) : 0.f;
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int r = (t >> 3) + 16 * k, c = (t & 7) * 16;
    if (r < r0 || r >= r1) continue;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack_codes<CODE>(bf_lo(x[k][2 * i]) * inv, bf_hi(x[k][2 * i]) * inv, bf_lo(x[k][2 * i + 1]) * inv,
                              bf_hi(x[k][2 * i + 1]) * inv);
    *reinterpret_cast<uint4*>(codes + r * kD + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (r0 > 0 && s > before) {   // the page's earlier rows under the larger scale
    const float ratio = before * inv;
    for (int e = t; e < r0 * 8; e += 128) {
      uint4* at = reinterpret_cast<uint4*>(codes) + e;
      const uint4 v = *at;
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        codes_f32<CODE>(in[i], f);
        o[i] = pack_codes<CODE>(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
      }
      *at = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
  if (t == 0) *scale = s;
}

struct ReadParams {
  lrkv_paged_dims D;
  lrkv_paged_cache C;
  const int32_t* first;
  const int32_t* count;
  lrkv_bf16* k_out;
  lrkv_bf16* v_out;
  int layer, t_max;
  int out32;   // 32-byte stores allowed
};

constexpr int kReadThreads = 256, kReadRows = 64;   // rows per CTA: two per group of eight threads

template <int CODE>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const lrkv_paged_dims& D = p.D;
  const int h = blockIdx.x % D.Hkv, i0 = blockIdx.x / D.Hkv * kReadRows, b = blockIdx.y;
  uint32_t status = 0;
  const int n = call_tokens(p.count, b, p.t_max, &status);
  const int base = p.first ? p.first[b] : 0;
  const long long cap = (long long)D.max_pages * D.page;
  if (n > 0 && (base < 0 || (long long)base + n > cap)) status |= LRKV_DEV_SEQ_OVERFLOW;
  if (status && h == 0 && i0 == 0 && threadIdx.x == 0) atomicOr(p.C.dev_status, status);
  const int c = (threadIdx.x & 7) * 16;
  uint4 in[2][2];
  float sc[2][2];
  bool ok[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int i = i0 + (threadIdx.x >> 3) + 32 * q;
    const long long pos = (long long)base + i;
    ok[q] = i < n && pos >= 0 && pos < cap;
    if (!ok[q]) continue;
    const int slot = (int)(pos / D.page), r = (int)(pos % D.page);
    const int pid = p.C.page_table[(size_t)b * D.max_pages + slot];
    if (pid < 0 || pid >= D.n_pages) {
      ok[q] = false;
      if (c == 0) atomicOr(p.C.dev_status, LRKV_DEV_BAD_PAGE);
      continue;
    }
    const size_t ph = ((size_t)p.layer * D.n_pages + pid) * D.Hkv + h;
    const size_t at = (ph * D.page + r) * kD + c;
    in[q][0] = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.C.k) + at);
    in[q][1] = *reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.C.v) + at);
    sc[q][0] = p.C.scale_k[ph];
    sc[q][1] = p.C.scale_v[ph];
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (!ok[q]) continue;
    const int i = i0 + (threadIdx.x >> 3) + 32 * q;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint4 v = in[q][side];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      const float s = sc[q][side];
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[4];
        codes_f32<CODE>(w[k], f);
        o[2 * k] = cvt_bf16x2(f[0] * s, f[1] * s);
        o[2 * k + 1] = cvt_bf16x2(f[2] * s, f[3] * s);
      }
      uint4* dst = reinterpret_cast<uint4*>((side == 0 ? p.k_out : p.v_out) +
                                            (((size_t)b * p.t_max + i) * D.Hkv + h) * kD + c);
      if (p.out32) {   // whole sectors at a time
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]),
                     "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
      } else {
        __stcs(dst, make_uint4(o[0], o[1], o[2], o[3]));
        __stcs(dst + 1, make_uint4(o[4], o[5], o[6], o[7]));
      }
    }
  }
}

template <int CODE>
void (*append_for(int page))(const AppendParams) {
  switch (page) {
    case 16: return append_kernel<16, CODE>;
    case 32: return append_kernel<32, CODE>;
    case 64: return append_kernel<64, CODE>;
    default: return append_kernel<128, CODE>;
  }
}

}  // namespace paged
}  // namespace lrkv

using namespace lrkv;

extern "C" {

lrkv_status lrkv_paged_append(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, int32_t layer,
                              const lrkv_bf16* k_new, const lrkv_bf16* v_new, int32_t t_new,
                              const int32_t* t_new_b, void* stream) {
  lrkv_status st = paged::check_all(dims, cache);
  if (st != LRKV_OK) return st;
  if (layer < 0 || layer >= dims->n_layers || t_new < 0) return LRKV_ERR_INVALID_ARG;
  if (t_new > (1 << 24)) return LRKV_ERR_UNSUPPORTED;
  if (t_new == 0) return LRKV_OK;
  if (!k_new || !v_new) return LRKV_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(t_new_b)) return LRKV_ERR_ALIGNMENT;
  paged::AppendParams p = {};
  p.D = *dims;
  p.C = *cache;
  p.k_new = k_new;
  p.v_new = v_new;
  p.t_new_b = t_new_b;
  p.layer = layer;
  p.t_new = t_new;
  p.touched = (t_new + dims->page - 2) / dims->page + 1;
  const long long gx = (long long)p.touched * dims->Hkv;
  if (gx >= (1LL << 31)) return LRKV_ERR_UNSUPPORTED;
  auto kern = dims->code == LRKV_CODE_INT8 ? paged::append_for<LRKV_CODE_INT8>(dims->page)
                                           : paged::append_for<LRKV_CODE_E4M3>(dims->page);
  return launch_pdl(kern, dim3((unsigned)gx, dims->B), dim3(paged::kAppendThreads), 0,
                    static_cast<cudaStream_t>(stream), p);
}

lrkv_status lrkv_paged_read(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, int32_t layer,
                            const int32_t* first, const int32_t* count, int32_t t_max, lrkv_bf16* k_out,
                            lrkv_bf16* v_out, void* stream) {
  lrkv_status st = paged::check_all(dims, cache);
  if (st != LRKV_OK) return st;
  if (layer < 0 || layer >= dims->n_layers || t_max < 0) return LRKV_ERR_INVALID_ARG;
  if (t_max > (1 << 24)) return LRKV_ERR_UNSUPPORTED;
  if (t_max == 0) return LRKV_OK;
  if (!count || !k_out || !v_out) return LRKV_ERR_INVALID_ARG;
  if (!aligned16(first) || !aligned16(count) || !aligned16(k_out) || !aligned16(v_out)) return LRKV_ERR_ALIGNMENT;
  paged::ReadParams p = {};
  p.D = *dims;
  p.C = *cache;
  p.first = first;
  p.count = count;
  p.k_out = k_out;
  p.v_out = v_out;
  p.layer = layer;
  p.t_max = t_max;
  p.out32 = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  const long long gx = (long long)((t_max + paged::kReadRows - 1) / paged::kReadRows) * dims->Hkv;
  if (gx >= (1LL << 31)) return LRKV_ERR_UNSUPPORTED;
  auto kern = dims->code == LRKV_CODE_INT8 ? paged::read_kernel<LRKV_CODE_INT8> : paged::read_kernel<LRKV_CODE_E4M3>;
  return launch_pdl(kern, dim3((unsigned)gx, dims->B), dim3(paged::kReadThreads), 0,
                    static_cast<cudaStream_t>(stream), p);
}

}  // extern "C"
