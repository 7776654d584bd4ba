// lrkv_prefill_attn: argument checks, tensor maps and the launch.
#include "prefill_attn.cuh"

#include "../launch_util.cuh"
#include "serve_host.cuh"
#include "tensor_map.cuh"

namespace {

using namespace lrkv;

// Rows [B][t][H][128] as a 4-d tensor (128, H, t, B): boxes of 64 columns x 1 head
// x 64 tokens, 128-byte swizzle, zeros past the last token of a batch row.
bool rows_map(CUtensorMap* map, const lrkv_bf16* base, int B, int t, int H, const int64_t (&st)[3]) {
  serve::EncodeTiledFn enc = serve::encode_tiled();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)H, (cuuint64_t)t, (cuuint64_t)B};
  // a stride whose extent is 1 is never used: any valid number does
  const cuuint64_t sh = H > 1 ? (cuuint64_t)st[2] * 2 : (cuuint64_t)kD * 2;
  const cuuint64_t stt = t > 1 ? (cuuint64_t)st[1] * 2 : (cuuint64_t)kD * 2;
  const cuuint64_t sb = B > 1 ? (cuuint64_t)st[0] * 2 : (cuuint64_t)kD * 2;
  const cuuint64_t strides[3] = {sh, stt, sb};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)prefill::kUnit, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<lrkv_bf16*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool strides_ok(const int64_t (&st)[3], int B, int t, int H) {
  const int ext[3] = {B, t, H};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] <= 1) continue;
    if (st[i] <= 0 || st[i] % 8 != 0 || st[i] >= (1LL << 38)) return false;
  }
  return true;
}

lrkv_status check(const lrkv_prefill_dims* D) {
  if (!D || D->B < 1 || D->Hq < 1 || D->Hkv < 1 || D->t_q < 0 || D->t_k < 0) return LRKV_ERR_INVALID_ARG;
  if (D->Hq % D->Hkv) return LRKV_ERR_INVALID_ARG;
  if (D->d != kD || D->B > 65535 || D->Hq > 65535) return LRKV_ERR_UNSUPPORTED;
  if (D->t_q > (1 << 24) || D->t_k > (1 << 24)) return LRKV_ERR_UNSUPPORTED;   // positions in fp32
  if (!strides_ok(D->q_stride, D->B, D->t_q, D->Hq) || !strides_ok(D->out_stride, D->B, D->t_q, D->Hq) ||
      !strides_ok(D->k_stride, D->B, D->t_k, D->Hkv) || !strides_ok(D->v_stride, D->B, D->t_k, D->Hkv))
    return LRKV_ERR_INVALID_ARG;
  const long long blocks = ((long long)D->t_q + 2 * prefill::kTile - 1) / (2 * prefill::kTile);
  if (blocks * D->Hq * D->B >= (1LL << 31)) return LRKV_ERR_UNSUPPORTED;
  return LRKV_OK;
}

// CTAs that share the keys of a pair of query blocks: one where the blocks fill the SMs;
// else as many as fill them, with 6 units of keys for each at least, as a CTA's start and end
// cost as much as 7 units and the join takes a launch.  (100 rows x 4 heads after 8000 keys:
// 115 us in one piece, 21 us with 6 units at least, 23 with 8, 26 with 4.)
int splits(const lrkv_prefill_dims& D) {
  const long long ctas = ((long long)D.t_q + 2 * prefill::kTile - 1) / (2 * prefill::kTile) * D.Hq * D.B;
  if (ctas == 0) return 1;
  long long n = num_sms() / ctas;
  const long long most = D.t_k / (6 * prefill::kUnit);
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

}  // namespace

extern "C" {

size_t lrkv_prefill_workspace_size(const lrkv_prefill_dims* dims) {
  if (check(dims) != LRKV_OK) return 0;
  const int n = splits(*dims);
  return n > 1 ? (size_t)n * dims->B * dims->Hq * dims->t_q * prefill::kPart * sizeof(float) : 0;
}

lrkv_status lrkv_prefill_attn(const lrkv_prefill_dims* dims, const lrkv_bf16* q, const lrkv_bf16* k,
                              const lrkv_bf16* v, const int32_t* q_len, const int32_t* kv_len,
                              const lrkv_score* score, lrkv_bf16* out, uint32_t* dev_status, void* ws,
                              size_t ws_bytes, void* stream) {
  lrkv_status st = check(dims);
  if (st != LRKV_OK) return st;
  if ((st = serve::check_score(score)) != LRKV_OK) return st;
  const lrkv_prefill_dims& D = *dims;
  if (D.t_q == 0) return LRKV_OK;
  if (!q || !out || (D.t_k > 0 && (!k || !v))) return LRKV_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, out, q_len, kv_len, dev_status, ws};
  for (const void* x : ptrs)
    if (!aligned16(x)) return LRKV_ERR_ALIGNMENT;
  prefill::Params p = {};
  p.n_split = splits(D);
  if (p.n_split > 1) {
    if (!ws || ws_bytes < lrkv_prefill_workspace_size(dims)) return LRKV_ERR_INVALID_ARG;
    p.part = static_cast<float*>(ws);
  }
  // no keys at all: the kernel writes zeros, its key and value maps are not used
  const int tk = D.t_k > 0 ? D.t_k : 1;
  if (!rows_map(&p.map_q, q, D.B, D.t_q, D.Hq, D.q_stride) ||
      !rows_map(&p.map_k, D.t_k > 0 ? k : q, D.t_k > 0 ? D.B : 1, tk, D.t_k > 0 ? D.Hkv : 1, D.k_stride) ||
      !rows_map(&p.map_v, D.t_k > 0 ? v : q, D.t_k > 0 ? D.B : 1, tk, D.t_k > 0 ? D.Hkv : 1, D.v_stride))
    return LRKV_ERR_CUDA;
  p.out = out;
  p.os_b = D.out_stride[0];
  p.os_t = D.out_stride[1];
  p.os_h = D.out_stride[2];
  p.q_len = q_len;
  p.kv_len = kv_len;
  p.dev_status = dev_status;
  p.B = D.B;
  p.Hq = D.Hq;
  p.Hkv = D.Hkv;
  p.t_q = D.t_q;
  p.t_k = D.t_k;
  p.n_blocks = (D.t_q + 2 * prefill::kTile - 1) / (2 * prefill::kTile);
  const serve::ScoreConsts sc = serve::score_consts(score);
  p.slopes = sc.slopes;
  p.first_key = sc.first_key;
  p.prefix_end = sc.prefix_end;
  p.window = sc.window;
  p.qk_log2 = sc.scale * kLog2e;
  const bool cap = sc.softcap > 0.f, bias = sc.slopes != nullptr;
  if (cap) {
    serve::cap_polynomial(sc.softcap, p.cap_poly);
    p.cap_unit = sc.scale / sc.softcap;
    p.cap_in = 2.f * kLog2e * sc.scale / sc.softcap;
    p.cap_log2 = sc.softcap * kLog2e;
  }
  p.out32 = (reinterpret_cast<uintptr_t>(out) & 31u) == 0 && (D.B == 1 || D.out_stride[0] % 16 == 0) &&
            (D.t_q == 1 || D.out_stride[1] % 16 == 0) && (D.Hq == 1 || D.out_stride[2] % 16 == 0);
  auto kern = cap ? (bias ? prefill::prefill_kernel<true, true> : prefill::prefill_kernel<true, false>)
                  : (bias ? prefill::prefill_kernel<false, true> : prefill::prefill_kernel<false, false>);
  if (!set_smem(kern, prefill::kSmemBytes)) return LRKV_ERR_CUDA;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const long long grid = (long long)p.n_blocks * D.Hq * D.B * p.n_split;
  st = launch_pdl(kern, dim3((unsigned)grid), dim3(prefill::kThreads), prefill::kSmemBytes, cs, p);
  if (st != LRKV_OK || p.n_split == 1) return st;
  const long long rows = (long long)D.B * D.Hq * D.t_q;
  return launch_pdl(prefill::join_kernel, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, cs, p);
}

}  // extern "C"
