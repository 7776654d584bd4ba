// lrkv_paged_attn: argument checks, tensor maps and the launch.
#include "paged_attn.cuh"

#include "../launch_util.cuh"
#include "tensor_map.cuh"

namespace {

using namespace lrkv;
using namespace lrkv::paged;

// All pages' codes as rows of 128 bytes; boxes of `rows` rows, 128-byte swizzle.
bool codes_map(CUtensorMap* map, void* base, uint64_t all_rows, int rows) {
  serve::EncodeTiledFn enc = serve::encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)all_rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kD};
  const cuuint32_t box[2] = {(cuuint32_t)kD, (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NB, int CODE, int PT>
lrkv_status launch(const AttnParams& p, int ctas, cudaStream_t s) {
  using C = AttnConfig<NB>;
  auto kern = p.cap_unit > 0.f || p.slopes ? attn_kernel<NB, CODE, PT, true> : attn_kernel<NB, CODE, PT, false>;
  if (!set_smem(kern, C::kSmem)) return LRKV_ERR_CUDA;
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(C::kThreads), C::kSmem, s, p);
}
template <int NB>
lrkv_status launch(const AttnParams& p, int ctas, cudaStream_t s) {
  if (p.D.code == LRKV_CODE_INT8)
    return p.D.page == 16 ? launch<NB, LRKV_CODE_INT8, 16>(p, ctas, s) : launch<NB, LRKV_CODE_INT8, 32>(p, ctas, s);
  return p.D.page == 16 ? launch<NB, LRKV_CODE_E4M3, 16>(p, ctas, s) : launch<NB, LRKV_CODE_E4M3, 32>(p, ctas, s);
}

}  // namespace

extern "C" {

size_t lrkv_paged_workspace_size(const lrkv_paged_dims* dims, int32_t t_q) {
  if (paged::check_dims(dims) != LRKV_OK || t_q < 1 || t_q > paged::kMaxTq) return 0;
  // enough for fewer rows too, which may pad to more than t_q does (32 rows fill one block, 36 two
  // of 24)
  size_t most = 0;
  for (int t = 1; t <= t_q; ++t) {
    const size_t n = paged::paged_ws(*dims, t).total;
    if (n > most) most = n;
  }
  return most;
}

lrkv_status lrkv_paged_attn(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, int32_t layer,
                            const lrkv_bf16* q, int32_t t_q, const int32_t* t_q_b, const lrkv_score* score,
                            lrkv_bf16* out, void* ws, size_t ws_bytes, void* stream) {
  lrkv_status st = paged::check_all(dims, cache);
  if (st != LRKV_OK) return st;
  if ((st = serve::check_score(score)) != LRKV_OK) return st;
  if (layer < 0 || layer >= dims->n_layers || t_q < 1) return LRKV_ERR_INVALID_ARG;
  if (t_q > paged::kMaxTq) return LRKV_ERR_UNSUPPORTED;
  if ((st = check_q_out(q, out)) != LRKV_OK) return st;
  if (!ws) return LRKV_ERR_INVALID_ARG;
  if (!aligned16(ws) || !aligned16(t_q_b)) return LRKV_ERR_ALIGNMENT;
  const PagedWs L = paged_ws(*dims, t_q);
  if (ws_bytes < L.total) return LRKV_ERR_INVALID_ARG;
  const uint64_t rows = (uint64_t)dims->n_layers * dims->n_pages * dims->Hkv * dims->page;
  if (rows >= (1ull << 31)) return LRKV_ERR_UNSUPPORTED;   // 32-bit tensor coordinates
  const uint64_t tiles = ((uint64_t)dims->max_pages * dims->page + paged::kTile - 1) / paged::kTile;
  if (tiles * dims->B * dims->Hkv * L.row_blocks >= (1ull << 31)) return LRKV_ERR_UNSUPPORTED;   // 32-bit tile numbers
  AttnParams p = {};
  const int box = dims->page < paged::kTile ? dims->page : paged::kTile;
  if (!codes_map(&p.map_k, cache->k, rows, box) || !codes_map(&p.map_v, cache->v, rows, box)) return LRKV_ERR_CUDA;
  p.D = *dims;
  p.C = *cache;
  p.q = q;
  p.out = out;
  p.t_q_b = t_q_b;
  const serve::ScoreConsts sc = serve::score_consts(score);
  p.slopes = sc.slopes;
  p.first_key = sc.first_key;
  p.prefix_end = sc.prefix_end;
  p.window = sc.window;
  p.row_log2 = sc.scale * kLog2e;
  if (sc.softcap > 0.f) {
    p.cap_unit = 1.f / (sc.softcap * kLog2e);
    serve::cap_polynomial(sc.softcap, p.cap_poly);
    p.cap_log2 = sc.softcap * kLog2e;
  }
  unsigned char* base = static_cast<unsigned char*>(ws);
  p.tickets = reinterpret_cast<int*>(base + L.tickets);
  p.recs = reinterpret_cast<float*>(base + L.recs);
  p.layer = layer;
  p.t_q = t_q;
  p.g = dims->Hq / dims->Hkv;
  p.row_blocks = L.row_blocks;
  p.per_block = (p.g * t_q + L.row_blocks - 1) / L.row_blocks;
  const uint32_t hr = (uint32_t)dims->Hkv * p.row_blocks;
  int ceil_log2 = 0;
  while ((1u << ceil_log2) < hr) ++ceil_log2;
  if (hr > 1) {   // exact for numbers below 2^31
    p.hr_mul = (uint32_t)(((1ull << (31 + ceil_log2)) + hr - 1) / hr);
    p.hr_shift = ceil_log2 - 1;
  }
  p.g_mul = 65536u / p.g + 1;
  p.page_shift = dims->page == 16 ? 4 : dims->page == 32 ? 5 : dims->page == 64 ? 6 : 7;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (L.rows) {
    case 8: return launch<1>(p, L.ctas, s);
    case 16: return launch<2>(p, L.ctas, s);
    case 24: return launch<3>(p, L.ctas, s);
    default: return launch<4>(p, L.ctas, s);
  }
}

}  // extern "C"
