/*
 * lrkv_serve.h -- C ABI of liblrkv_serve.so: the full-rank serving operators
 * that stand beside the low-rank cache of lrkv.h (NVIDIA B200, sm_100a).
 *
 *   lrkv_prefill_attn   attention of a prompt (or a chunk of one) over bf16
 *                       keys and values: what runs before lrkv_compress when a
 *                       prompt is prefilled at full rank (OjaKV repository
 *                       README, "OjaKV-PF": full-rank prefill attention, then
 *                       decode on the compressed cache)
 *   lrkv_paged_append   keys and values into a paged cache of 8-bit codes with
 *   lrkv_paged_read     one scale per page and head, and back to bf16 rows
 *   lrkv_paged_attn     attention of one or a few new tokens over that cache
 *   lrkv_pages_*        pages handed out, forked, freed, copied and compacted
 *
 * The paged 8-bit cache is for the layers (or the models) that a low-rank
 * basis does not fit: full rank at half the bytes of bf16.
 *
 * Conventions are those of lrkv.h: device pointers unless said otherwise, 16-byte
 * aligned, caller-owned; nothing is allocated, freed or synchronised; all work
 * is enqueued on `stream`; bad arguments are refused before any launch with
 * the status codes of lrkv.h; what only the device can see sets bits of the
 * status word.  Every call may be captured into a CUDA graph.  The current
 * device has to be the one that the stream and the pointers belong to.
 */
#ifndef LRKV_SERVE_H
#define LRKV_SERVE_H

#include "lrkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further bits of a status word (see LRKV_DEV_* in lrkv.h). */
#define LRKV_DEV_BAD_PAGE 0x10u  /* a page id outside [0, n_pages) where one was needed:
                                    its tokens were skipped (not written, not attended, not
                                    counted by lrkv_pages_advance) */
#define LRKV_DEV_NO_PAGES 0x20u  /* the pool ran out: the sequence (or fork) that did not
                                    fit, and those after it in the call, got nothing */
#define LRKV_DEV_BAD_SEQ 0x40u   /* a sequence index out of range or listed twice, a fork
                                    onto a sequence in use: that entry was skipped */

/* How scores are changed before the softmax, and which keys a row sees.  For the
 * query row at position i (counted over the whole sequence) and the key at j:
 *     s = scale q.k
 *     s = softcap tanh(s / softcap)            if softcap > 0
 *     s = s - slopes[head] |i - j|             if slopes
 *     seen: max(first_key, i - window + 1) <= j <= max(i, prefix_end - 1)
 * and j < the sequence's length.  A row that sees nothing gives zeros.  Keys that
 * are not seen may hold anything, NaN included; a row whose query or seen keys hold a NaN
 * gives NaN.  For what may lie in values that are not seen, see each call. */
typedef struct {
  float scale;               /* >= 0 and finite; 0 stands for 1 / sqrt(d) */
  float softcap;             /* >= 0 and finite; 0: none */
  int32_t window;            /* >= 0; 0: none */
  const float* slopes;       /* nullable [Hq]: distance bias (ALiBi), finite */
  const int32_t* first_key;  /* nullable [B][t_q]: the first key a row sees (the start of its
                                document); past the last one it may see: it sees nothing */
  const int32_t* prefix_end; /* nullable [B][t_q]: rows see every key below this, later
                                ones included (a bidirectional prefix); 0: causal */
} lrkv_score;

/* Sizes and strides of a prefill.  Strides are in elements, for {batch row,
 * token, head}; the d elements of one head of one token are contiguous.  Strides
 * of q, k, v and out are multiples of 8 and positive (any value where the extent
 * is 1); rows may so be slices of a fused projection's output. */
typedef struct {
  int32_t B, Hq, Hkv; /* Hq % Hkv == 0; query head h reads kv head h / (Hq / Hkv) */
  int32_t d;          /* 128 in this build */
  int32_t t_q, t_k;   /* query rows and keys per batch row (padded) */
  int64_t q_stride[3], k_stride[3], v_stride[3], out_stride[3];
} lrkv_prefill_dims;

/* Prefill attention: out = softmax(scores of lrkv_score) v, bf16 in and out.
 * Sequence b has kv_len[b] keys and q_len[b] query rows, which are its last
 * positions: row r is at i = kv_len[b] - q_len[b] + r (a first prompt has
 * q_len = kv_len; a later chunk has fewer rows than keys).
 *
 * q [B][t_q][Hq][d], k and v [B][t_k][Hkv][d], out [B][t_q][Hq][d], by strides.
 * q_len, kv_len: nullable [B] int32 (null: t_q, t_k); values outside the
 *   range are clamped into it (LRKV_DEV_BAD_COUNT).
 * Rows r >= q_len[b] of out are left as they were; rows of k and v at or past
 *   kv_len[b] are not used, whatever they hold.  Values below kv_len[b] have to
 *   be finite (a hidden key's value enters with weight zero).
 * out must not overlap q, k or v.
 * Scores and the softmax are in fp32; the weights are rounded to bf16 for the
 *   product with v, as v is bf16 (the sum that divides them is not).  Sums run up to
 *   2^24 times the weights' total: values have to stay below 2^80.
 * dev_status: nullable, 1 word of LRKV_DEV_* bits.
 * ws: lrkv_prefill_workspace_size(dims) bytes, any contents (0 bytes: may be
 *   null).  When there are few query rows the keys of a row block are split
 *   over several CTAs and their results joined from the workspace.
 */
LRKV_API size_t lrkv_prefill_workspace_size(const lrkv_prefill_dims* dims);
LRKV_API lrkv_status lrkv_prefill_attn(const lrkv_prefill_dims* dims, const lrkv_bf16* q,
                                       const lrkv_bf16* k, const lrkv_bf16* v,
                                       const int32_t* q_len, const int32_t* kv_len,
                                       const lrkv_score* score /* nullable: causal */,
                                       lrkv_bf16* out, uint32_t* dev_status, void* ws,
                                       size_t ws_bytes, void* stream);

/* ---- the paged 8-bit cache ------------------------------------------------ */

#define LRKV_CODE_INT8 0 /* symmetric integers in [-127, 127] */
#define LRKV_CODE_E4M3 1 /* 8-bit floats (e4m3, largest 448) */

typedef struct {
  int32_t B;         /* sequences (rows of the page table) */
  int32_t Hq, Hkv;   /* Hq % Hkv == 0, at most 8 query heads per kv head */
  int32_t d;         /* 128 in this build */
  int32_t page;      /* tokens per page: 16, 32, 64 or 128 */
  int32_t n_pages;   /* pages in the pool */
  int32_t max_pages; /* page table entries per sequence */
  int32_t n_layers;  /* layers that share the page table */
  int32_t code;      /* LRKV_CODE_* */
} lrkv_paged_dims;

/* One pool for all layers, one page table and one length per sequence: a page id
 * stands for the same tokens in every layer.  A page holds `page` tokens of every
 * kv head; its codes of one head share one scale: value = code * scale.  Scales are 0 or
 * 2^-100 and more, as lrkv_paged_append makes them. */
typedef struct {
  void* k;             /* [n_layers][n_pages][Hkv][page][d] bytes: codes */
  void* v;             /* likewise */
  float* scale_k;      /* [n_layers][n_pages][Hkv] */
  float* scale_v;      /* likewise */
  int32_t* page_table; /* [B][max_pages]: page ids of a sequence in order, -1: none */
  int32_t* seq_len;    /* [B] tokens in the cache */
  int32_t* refs;       /* [n_pages] sequences that hold the page; 0: free */
  uint32_t* dev_status; /* 1 word, LRKV_DEV_* bits */
} lrkv_paged_cache;
/* A new cache: page_table all -1, everything else zero.
 *
 * A step of a serving loop:
 *   lrkv_pages_reserve(t_new)                        pages for the new tokens
 *   per layer: lrkv_paged_append, lrkv_paged_attn    at positions seq_len ..
 *   lrkv_pages_advance(t_new)                        seq_len += t_new
 * and between steps lrkv_pages_fork / _free / _compact.  Only full pages are ever
 * shared between sequences, so an append never writes a shared page. */

/* Writes t_new tokens of every sequence at positions seq_len[b] .. of `layer`
 * (seq_len is not moved: lrkv_pages_advance does that once for all layers).
 *
 * k_new, v_new: [B][t_new][Hkv][d] bf16, dense; t_new_b: nullable [B] int32,
 *   tokens of each sequence (clamped into [0, t_new], LRKV_DEV_BAD_COUNT).
 * Per page and head, with Q = 127 or 448 and x the new elements on it (an
 * infinity counts as the largest finite bf16, a NaN as 0), all steps in fp32
 * with IEEE rounding:
 *     s   = max(scale of the page, max|x| / Q)   (0 for a page that starts with this call)
 *     s   = 0 if s < 2^-100
 *     inv = 1 / s  (0 if s = 0)
 *     code = x inv, rounded to the code's type (nearest, ties to even), in [-Q, Q]
 * and where s has grown, the codes already on the page are rounded once more:
 *     code = round(code (s_before inv)).
 * A page that starts with this call takes no account of what it held before.  Until then its
 * scale covers all that was appended to it, drafted tokens that were never advanced over
 * included: their effect on the scale, and on the codes that were rounded to it, stays.
 * Positions past the page table are dropped (LRKV_DEV_SEQ_OVERFLOW), as are
 * tokens whose table entry is no page (LRKV_DEV_BAD_PAGE). */
LRKV_API lrkv_status lrkv_paged_append(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                       int32_t layer, const lrkv_bf16* k_new,
                                       const lrkv_bf16* v_new, int32_t t_new,
                                       const int32_t* t_new_b, void* stream);

/* Reads positions first[b] .. first[b] + count[b] - 1 of `layer` back as bf16
 * (code * scale, rounded to fp32 and then to bf16): the keys and values that a later chunk of a prompt
 * attends to with lrkv_prefill_attn.
 * first: nullable [B] int32 (null: 0); count: [B] int32, clamped into [0, t_max].
 * k_out, v_out: [B][t_max][Hkv][d] bf16; rows at or past count[b], and rows
 * whose position has no page, are left as they were. */
LRKV_API lrkv_status lrkv_paged_read(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                     int32_t layer, const int32_t* first, const int32_t* count,
                                     int32_t t_max, lrkv_bf16* k_out, lrkv_bf16* v_out,
                                     void* stream);

/* Attention of t_q new tokens per sequence (1: a decode step; more: drafted
 * tokens being checked) over the pages of `layer`, causal among the new ones:
 * row r of sequence b is at position seq_len[b] + r and sees the keys that
 * `score` lets it see of positions 0 .. seq_len[b] + t_q_b[b] - 1 (append the
 * new tokens first).
 *
 * q: [B][t_q][Hq][d] bf16, dense; out: the same shape, bf16.
 * t_q_b: nullable [B] int32, rows of each sequence (clamped into [0, t_q]); rows
 *   past it are left as they were.
 * t_q: 1 .. 64.
 * ws: lrkv_paged_workspace_size(dims, t_q) bytes (for this t_q or a larger one),
 *   zero-filled once; the calls leave it as they need it.  A workspace belongs to one
 *   lrkv_paged_dims (another lays it out in another way) and serves one stream of calls (two
 *   captured graphs that may run at the same time need one each).
 * LRKV_ERR_UNSUPPORTED for a pool of 2^31 rows of codes or more, or a page table with
 *   room for 2^31 tiles of 32 tokens over all sequences, kv heads and blocks of query rows.
 * Logits and softmax in fp32; queries and weights enter the products as f16
 * (queries scaled by a power of two: exact up to 2^-28 of the row's largest
 * element; weights rounded to 11 bits down to 2^-21 of the row's largest, to steps of at
 * most 2^-31 of it below that; the sum that divides them is not rounded).  int8 codes
 * enter the fp32 sums with 128 added, which is taken off again.  A value that a mask hides
 * enters with weight zero and has to be finite (the e4m3 codes 0x7f and 0xff are NaN;
 * lrkv_paged_append writes neither). */
LRKV_API size_t lrkv_paged_workspace_size(const lrkv_paged_dims* dims, int32_t t_q);
LRKV_API lrkv_status lrkv_paged_attn(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                     int32_t layer, const lrkv_bf16* q, int32_t t_q,
                                     const int32_t* t_q_b, const lrkv_score* score,
                                     lrkv_bf16* out, void* ws, size_t ws_bytes, void* stream);

/* ---- pages ------------------------------------------------------------------
 * Free pages are those with refs = 0; they are handed out lowest id first, in
 * the order of the sequences (or list entries) that ask.  A sequence's row of the
 * page table is filled from the front.  Lists of sequences have at most 2^16 entries, lists of
 * pages 2^24 (LRKV_ERR_UNSUPPORTED beyond).  ws: the
 * workspace of lrkv_paged_attn (any t_q). */

/* Pages for t_new (or t_new_b[b]) more tokens of every sequence.  A sequence for
 * which the pool, or its row of the page table, does not suffice gets none, nor do
 * those after it where the pool ran out (LRKV_DEV_NO_PAGES, LRKV_DEV_SEQ_OVERFLOW). */
LRKV_API lrkv_status lrkv_pages_reserve(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                        int32_t t_new, const int32_t* t_new_b, void* stream);

/* seq_len[b] += t_new (or t_new_b[b]), at most max_pages * page (LRKV_DEV_SEQ_OVERFLOW) and
 * never over a token whose table entry is no page: a sequence to which lrkv_pages_reserve gave
 * nothing stops in front of its first such token (LRKV_DEV_BAD_PAGE). */
LRKV_API lrkv_status lrkv_pages_advance(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                        int32_t t_new, const int32_t* t_new_b, void* stream);

/* Sequence dst[i] becomes a copy of sequence src[i], for i < n: full pages are
 * shared, a last page that is not full is copied (all layers) to a page of its own.
 * dst[i] has to be empty (seq_len 0 and no pages), and is named once (of entries that
 * name it again the first counts, LRKV_DEV_BAD_SEQ); a source may be named many times.
 * Sources are taken as they were before the call; an entry whose source has no page for its
 * last tokens is skipped (LRKV_DEV_BAD_PAGE).
 * src, dst: device [n] int32. */
LRKV_API lrkv_status lrkv_pages_fork(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                     const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                                     size_t ws_bytes, void* stream);

/* Empties the sequences seqs[0..n-1] (device int32): their pages lose a reference,
 * their table rows become -1, their lengths 0.  An index listed twice counts once
 * (LRKV_DEV_BAD_SEQ). */
LRKV_API lrkv_status lrkv_pages_free(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                     const int32_t* seqs, int32_t n, void* stream);

/* Copies pages src[i] to dst[i] (device [n] int32) in every layer, codes and
 * scales.  All dst have to be different, and none of them a src: of entries that
 * break this the first to name a dst wins, an entry whose src is some entry's dst
 * is skipped, and LRKV_DEV_BAD_PAGE is set; as for ids out of range.  refs and the
 * page table stay as they are. */
LRKV_API lrkv_status lrkv_pages_copy(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache,
                                     const int32_t* src, const int32_t* dst, int32_t n, void* ws,
                                     size_t ws_bytes, void* stream);

/* Moves pages so that the live ones are 0 .. (live - 1): the i-th live page at or
 * behind that border, by id, goes to the i-th free page before it.  Page table
 * and refs follow. */
LRKV_API lrkv_status lrkv_pages_compact(const lrkv_paged_dims* dims,
                                        const lrkv_paged_cache* cache, void* ws, size_t ws_bytes,
                                        void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LRKV_SERVE_H */
