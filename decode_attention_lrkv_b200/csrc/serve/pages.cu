// lrkv_pages_*: pages handed out, forked, freed, copied and compacted.
//
// What orders pages (which free page goes to whom, which entry of a list comes
// first) is decided by one CTA with prefix sums, so results do not depend on how
// threads run; what moves bytes (whole pages of every layer, table rows) is spread
// over the GPU by a second kernel that reads those decisions from the workspace.
// Bound by memory: every moved page is read and written once.
#include "paged.cuh"

#include "../launch_util.cuh"

namespace lrkv {
namespace paged {

constexpr int kPlanThreads = 1024, kMoveThreads = 256;
constexpr int kMoveVec = 4;   // 16-byte pieces that a thread has in flight
constexpr int kMoveBytes = kMoveThreads * kMoveVec * 16;
// Entries of a list of sequences.  There are 65535 sequences at most, so a longer one names some of
// them twice; to find those, an entry is compared with all before it (2^31 comparisons for such a
// list, a few ms of the whole GPU; for 2^24 entries it would be minutes).
constexpr int kMaxSeqList = 1 << 16;

struct PageParams {
  lrkv_paged_dims D;
  lrkv_paged_cache C;
  const int32_t* src;       // fork, copy: lists; free: seqs
  const int32_t* dst;
  const int32_t* t_new_b;
  int n, t_new;
  int* claims;              // zero between calls
  int* ticket;              // likewise
  int* list;                // [0]: pages to move; [4 ..): their sources, then from `half` their targets
  int half;                 // max(n_pages, B)
};

__device__ __forceinline__ bool in_range(int v, int n) { return v >= 0 && v < n; }

// Exclusive prefix sum over the block; *total: the sum (in every thread).
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += u;
  }
  __syncthreads();   // earlier readers of warp_sums are done
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[kPlanThreads / 32 - 1];
  return (warp ? warp_sums[warp - 1] : 0) + sum - v;
}

// Four consecutive reference counts from page i (i % 4 == 0); -1 past the pool.
__device__ __forceinline__ int4 refs4(const PageParams& p, int i) {
  if (i + 3 < p.D.n_pages) return *reinterpret_cast<const int4*>(p.C.refs + i);
  int4 r = make_int4(-1, -1, -1, -1);
  if (i < p.D.n_pages) r.x = p.C.refs[i];
  if (i + 1 < p.D.n_pages) r.y = p.C.refs[i + 1];
  if (i + 2 < p.D.n_pages) r.z = p.C.refs[i + 2];
  return r;
}

// Calls take(rank, page) for the lowest free pages, rank from 0, until `want` are
// found; returns how many there are, at most `want`.
template <typename Take>
__device__ __forceinline__ int free_pages(const PageParams& p, int want, int* warp_sums, Take take) {
  int found = 0;
  for (int i0 = 0; i0 < p.D.n_pages && found < want; i0 += 4 * kPlanThreads) {
    const int i = i0 + 4 * threadIdx.x;
    const int4 r = refs4(p, i);
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    int total;
    int rank = found + block_scan(f[0] + f[1] + f[2] + f[3], warp_sums, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) {
        if (rank < want) take(rank, i + k);
        ++rank;
      }
    found = min(want, found + total);
  }
  return found;
}

// ---- reserve, advance -------------------------------------------------------------

// Pages that sequence b lacks for its new tokens; *slot: the first such slot of its row.
__device__ __forceinline__ int lacking(const PageParams& p, int b, int* slot, uint32_t* status) {
  const int n = call_tokens(p.t_new_b, b, p.t_new, status);
  const long long cap = (long long)p.D.max_pages * p.D.page;
  const int len = (int)min((long long)max(p.C.seq_len[b], 0), cap);
  if (n == 0) return 0;
  if (len + (long long)n > cap) {
    *status |= LRKV_DEV_SEQ_OVERFLOW;
    return 0;
  }
  const int stop = (int)((len + (long long)n + p.D.page - 1) / p.D.page);
  int s = len / p.D.page;
  while (s < stop && p.C.page_table[(size_t)b * p.D.max_pages + s] >= 0) ++s;
  *slot = s;
  return stop - s;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const __grid_constant__ PageParams p) {
  __shared__ int warp_sums[32], off[kPlanThreads + 1], first[kPlanThreads];
  __shared__ int s_stop;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  uint32_t status = 0;
  long long want = 0;   // pages of all sequences
  for (int b0 = 0; b0 < p.D.B; b0 += kPlanThreads) {
    int slot, total;
    const int need = b0 + tid < p.D.B ? lacking(p, b0 + tid, &slot, &status) : 0;
    block_scan(need, warp_sums, &total);
    want += total;
  }
  if (status) atomicOr(p.C.dev_status, status);
  if (want == 0) return;
  // pages there are, at most as many as are wanted
  const int have = free_pages(p, (int)min(want, (long long)p.D.n_pages), warp_sums, [](int, int) {});
  int given = 0;
  for (int b0 = 0; b0 < p.D.B; b0 += kPlanThreads) {
    int slot = 0, total;
    const int need = b0 + tid < p.D.B ? lacking(p, b0 + tid, &slot, &status) : 0;
    const int before = block_scan(need, warp_sums, &total);
    if (tid == 0) s_stop = 0x7fffffff, off[kPlanThreads] = total;
    off[tid] = before;
    first[tid] = slot;
    __syncthreads();
    // the pool ends before this sequence has all it wants: it and those after it get none
    const bool out = need > 0 && (long long)given + before + need > have;
    if (out) atomicMin(&s_stop, before), status |= LRKV_DEV_NO_PAGES;
    __syncthreads();
    const int stop = min(s_stop, total);
    free_pages(p, stop, warp_sums, [&](int rank, int page) {
      int lo = 0, hi = kPlanThreads;   // the last sequence with off <= rank that wants pages
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= rank) lo = mid; else hi = mid;
      }
      p.C.page_table[(size_t)(b0 + lo) * p.D.max_pages + first[lo] + rank - off[lo]] = page;
      p.C.refs[page] = 1;
    });
    given += stop;
    const bool ended = s_stop != 0x7fffffff;
    __syncthreads();
    if (ended) break;
  }
  if (status) atomicOr(p.C.dev_status, status);
}

// A warp per sequence: its lanes look through the table entries that the new tokens need, all of
// them (no early end, so the loads do not wait for one another).
__global__ void __launch_bounds__(kMoveThreads) advance_kernel(const __grid_constant__ PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (b >= p.D.B) return;
  uint32_t status = 0;
  const int n = call_tokens(p.t_new_b, b, p.t_new, &status);
  const int cap = p.D.max_pages * p.D.page;
  const int len = min(max(p.C.seq_len[b], 0), cap);
  if (len + n > cap) status |= LRKV_DEV_SEQ_OVERFLOW;
  int stop = min(len + n, cap);
  // the first slot that has no page: the tokens from there on were never stored
  const int* row = p.C.page_table + (size_t)b * p.D.max_pages;
  const int end = (stop + p.D.page - 1) / p.D.page;
  int hole = end;
  if (stop > len)
#pragma unroll 16
    for (int s = len / p.D.page + lane; s < end; s += 32)
      if (!in_range(row[s], p.D.n_pages)) hole = min(hole, s);
  hole = __reduce_min_sync(0xffffffffu, hole);
  if (hole < end) status |= LRKV_DEV_BAD_PAGE, stop = max(len, hole * p.D.page);
  if (lane != 0) return;
  p.C.seq_len[b] = stop;
  if (status) atomicOr(p.C.dev_status, status);
}

// ---- moving whole pages -------------------------------------------------------------

// One thread block's part of a page copy: piece `piece` of keys and values of (layer, pair).
__device__ __forceinline__ void move_piece(const PageParams& p, int layer, int from, int to, int piece) {
  const size_t elems = page_elems(p.D);
  const size_t a = ((size_t)layer * p.D.n_pages + from), b = ((size_t)layer * p.D.n_pages + to);
  const size_t at = (size_t)piece * kMoveBytes;
  uint4 x[2][kMoveVec];
  const unsigned char* const src[2] = {static_cast<const unsigned char*>(p.C.k) + a * elems,
                                       static_cast<const unsigned char*>(p.C.v) + a * elems};
  unsigned char* const dst[2] = {static_cast<unsigned char*>(p.C.k) + b * elems,
                                 static_cast<unsigned char*>(p.C.v) + b * elems};
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int k = 0; k < kMoveVec; ++k) {
      const size_t o = at + ((size_t)k * kMoveThreads + threadIdx.x) * 16;
      if (o < elems) x[side][k] = __ldcs(reinterpret_cast<const uint4*>(src[side] + o));
    }
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int k = 0; k < kMoveVec; ++k) {
      const size_t o = at + ((size_t)k * kMoveThreads + threadIdx.x) * 16;
      if (o < elems) __stcs(reinterpret_cast<uint4*>(dst[side] + o), x[side][k]);
    }
  if (piece == 0)
    for (int h = threadIdx.x; h < p.D.Hkv; h += kMoveThreads) {
      p.C.scale_k[b * p.D.Hkv + h] = p.C.scale_k[a * p.D.Hkv + h];
      p.C.scale_v[b * p.D.Hkv + h] = p.C.scale_v[a * p.D.Hkv + h];
    }
}
__device__ __forceinline__ int move_pieces(const PageParams& p) {
  return (int)((page_elems(p.D) + kMoveBytes - 1) / kMoveBytes);
}
// All layers of the listed pages, spread over the grid.
__device__ __forceinline__ void move_listed(const PageParams& p) {
  const int n = p.list[0], pieces = move_pieces(p);
  const long long items = (long long)n * p.D.n_layers * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = (int)(it % pieces);
    const long long rest = it / pieces;
    const int i = (int)(rest % n), layer = (int)(rest / n);
    move_piece(p, layer, p.list[4 + i], p.list[4 + p.half + i], piece);
  }
}

// ---- fork --------------------------------------------------------------------------
// The plan, for every sequence b: from[b] = 1 + the sequence that b becomes a copy of (0:
// none), len[b] its length, own[b] = 1 + the place of b's own last page in the list of
// pages to move (0: it has none).

__device__ __forceinline__ int* list_part(const PageParams& p, int k) { return p.list + 4 + (size_t)k * p.half; }

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const __grid_constant__ PageParams p) {
  __shared__ int warp_sums[32];
  __shared__ int s_stop;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int *source = list_part(p, 0), *target = list_part(p, 1), *from = list_part(p, 2), *len = list_part(p, 3),
      *own = list_part(p, 4);
  uint32_t status = 0;
  for (int b = tid; b < p.D.B; b += kPlanThreads) from[b] = 0;
  for (int i = tid; i < p.n; i += kPlanThreads)
    if (in_range(p.dst[i], p.D.B)) atomicMax(p.claims + p.dst[i], 0x7fffffff - i);   // the first to name it
  if (tid == 0) s_stop = 0x7fffffff;
  __syncthreads();
  // which entries hold, and the pages of their own that they want
  int want = 0;
  for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
    const int i = i0 + tid;
    bool part = false;
    int s = -1, d = -1, T = 0, page = -1;
    if (i < p.n) {
      s = p.src[i];
      d = p.dst[i];
      if (in_range(s, p.D.B) && in_range(d, p.D.B) && s != d && p.claims[d] == 0x7fffffff - i &&
          p.C.seq_len[d] == 0 && p.C.page_table[(size_t)d * p.D.max_pages] < 0) {
        T = min(max(p.C.seq_len[s], 0), p.D.max_pages * p.D.page);
        if (T % p.D.page) {
          page = p.C.page_table[(size_t)s * p.D.max_pages + T / p.D.page];
          part = in_range(page, p.D.n_pages);
          if (!part) status |= LRKV_DEV_BAD_PAGE, d = -1;   // the source's own last tokens are not there
        }
      } else {
        status |= LRKV_DEV_BAD_SEQ;
        d = -1;
      }
    }
    int total;
    const int rank = want + block_scan(part, warp_sums, &total);
    if (part) source[rank] = page;
    if (d >= 0) {
      from[d] = s + 1;
      len[d] = T;
      own[d] = part ? rank + 1 : 0;
    }
    want += total;
  }
  __syncthreads();
  const int have = free_pages(p, want, warp_sums, [&](int rank, int page) { target[rank] = page; });
  __syncthreads();
  if (have < want) {   // the first entry whose page the pool does not hold: it and those after it get nothing
    for (int i = tid; i < p.n; i += kPlanThreads) {
      const int d = p.dst[i];
      if (in_range(d, p.D.B) && p.claims[d] == 0x7fffffff - i && from[d] && own[d] == have + 1) s_stop = i;
    }
    __syncthreads();
    for (int i = tid; i < p.n; i += kPlanThreads) {
      const int d = p.dst[i];
      if (i >= s_stop && in_range(d, p.D.B) && p.claims[d] == 0x7fffffff - i && from[d])
        from[d] = 0, status |= LRKV_DEV_NO_PAGES;
    }
  }
  __syncthreads();
  for (int r = tid; r < have; r += kPlanThreads) p.C.refs[target[r]] = 1;
  for (int i = tid; i < p.n; i += kPlanThreads)
    if (in_range(p.dst[i], p.D.B)) p.claims[p.dst[i]] = 0;
  if (tid == 0) p.list[0] = have;
  if (status) atomicOr(p.C.dev_status, status);
}

__global__ void __launch_bounds__(kMoveThreads) fork_move_kernel(const __grid_constant__ PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int *target = list_part(p, 1), *from = list_part(p, 2), *len = list_part(p, 3), *own = list_part(p, 4);
  move_listed(p);
  // table rows: entries of full pages, then the page of its own
  for (int i = (int)blockIdx.x; i < p.n; i += gridDim.x) {
    const int d = p.dst[i];
    // an entry that did not hold has another source than the plan's, or is a second one with the same
    // source: it writes the same row, so the references are counted by the first one alone
    if (!in_range(d, p.D.B) || from[d] == 0 || from[d] != p.src[i] + 1) continue;
    bool first = true;
    for (int j = threadIdx.x; j < i; j += kMoveThreads) first &= p.dst[j] != d;
    if (!__syncthreads_and(first)) continue;
    const int* src = p.C.page_table + (size_t)p.src[i] * p.D.max_pages;
    int* dst = p.C.page_table + (size_t)d * p.D.max_pages;
    const int full = len[d] / p.D.page;
    uint32_t status = 0;
    for (int k = threadIdx.x; k < full; k += kMoveThreads) {
      const int page = src[k];
      dst[k] = page;
      if (in_range(page, p.D.n_pages)) atomicAdd(p.C.refs + page, 1);
      else status |= LRKV_DEV_BAD_PAGE;
    }
    if (threadIdx.x == 0) {
      if (own[d]) dst[full] = target[own[d] - 1];
      p.C.seq_len[d] = len[d];
    }
    if (status) atomicOr(p.C.dev_status, status);
  }
}

// ---- free --------------------------------------------------------------------------

__global__ void __launch_bounds__(kMoveThreads) free_kernel(const __grid_constant__ PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  for (int i = (int)blockIdx.x; i < p.n; i += gridDim.x) {
    const int b = p.src[i];
    bool first = in_range(b, p.D.B);
    for (int j = threadIdx.x; first && j < i; j += kMoveThreads) first = p.src[j] != b;
    if (!__syncthreads_and(first)) {
      if (threadIdx.x == 0) atomicOr(p.C.dev_status, LRKV_DEV_BAD_SEQ);
      continue;
    }
    int* row = p.C.page_table + (size_t)b * p.D.max_pages;
    uint32_t status = 0;
    for (int k = threadIdx.x; k < p.D.max_pages; k += kMoveThreads) {
      const int page = row[k];
      if (page == -1) continue;
      row[k] = -1;
      if (!in_range(page, p.D.n_pages)) {
        status |= LRKV_DEV_BAD_PAGE;
        continue;
      }
      if (atomicSub(p.C.refs + page, 1) <= 0) {   // nobody held it: leave the count as it was
        atomicAdd(p.C.refs + page, 1);
        status |= LRKV_DEV_BAD_PAGE;
      }
    }
    if (threadIdx.x == 0) p.C.seq_len[b] = 0;
    if (status) atomicOr(p.C.dev_status, status);
  }
}

// ---- copy --------------------------------------------------------------------------

__global__ void copy_claim_kernel(const __grid_constant__ PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= p.n) return;
  if (in_range(p.dst[i], p.D.n_pages)) atomicMax(p.claims + p.dst[i], 0x7fffffff - i);   // the first to name it
  else atomicOr(p.C.dev_status, LRKV_DEV_BAD_PAGE);
}
__global__ void __launch_bounds__(kMoveThreads) copy_move_kernel(const __grid_constant__ PageParams p) {
  __shared__ int s_last;
  griddep_wait();
  griddep_launch_dependents();
  const int pieces = move_pieces(p);
  const long long items = (long long)p.n * p.D.n_layers * pieces;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = (int)(it % pieces);
    const long long rest = it / pieces;
    const int i = (int)(rest % p.n), layer = (int)(rest / p.n);
    const int from = p.src[i], to = p.dst[i];
    if (!in_range(to, p.D.n_pages)) continue;
    if (!in_range(from, p.D.n_pages) || p.claims[to] != 0x7fffffff - i || p.claims[from] != 0) {
      if (piece == 0 && layer == 0 && threadIdx.x == 0) atomicOr(p.C.dev_status, LRKV_DEV_BAD_PAGE);
      continue;
    }
    move_piece(p, layer, from, to, piece);
  }
  // the last CTA clears the claims
  __syncthreads();
  if (threadIdx.x == 0) s_last = atom_add_acq_rel_gpu(p.ticket, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  for (int i = threadIdx.x; i < p.n; i += kMoveThreads)
    if (in_range(p.dst[i], p.D.n_pages)) p.claims[p.dst[i]] = 0;
  if (threadIdx.x == 0) *p.ticket = 0;
}

// ---- compact ------------------------------------------------------------------------

// Lists: the live pages at or behind the border and the free ones before it, as many of
// each; place[i]: page i's place in the first list (unset for pages that are not in it).
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ PageParams p) {
  __shared__ int warp_sums[32];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  int *source = list_part(p, 0), *target = list_part(p, 1), *place = list_part(p, 2);
  int live = 0;
  {
    int n = 0, total;
    for (int i = 4 * tid; i < p.D.n_pages; i += 4 * kPlanThreads) {
      const int4 r = refs4(p, i);
      n += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    }
    block_scan(n, warp_sums, &total);
    live = total;
  }
  int holes = 0;
  for (int i0 = 0; i0 < live; i0 += 4 * kPlanThreads) {
    const int i = i0 + 4 * tid;
    const int4 r = refs4(p, i);
    const int f[4] = {r.x <= 0 && i < live, r.y <= 0 && i + 1 < live, r.z <= 0 && i + 2 < live, r.w <= 0 && i + 3 < live};
    int total;
    int rank = holes + block_scan(f[0] + f[1] + f[2] + f[3], warp_sums, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) target[rank++] = i + k;
    holes += total;
  }
  __syncthreads();
  int found = 0;
  for (int i0 = live / 4 * 4; i0 < p.D.n_pages; i0 += 4 * kPlanThreads) {
    const int i = i0 + 4 * tid;
    const int4 r = refs4(p, i);
    const int f[4] = {r.x > 0 && i >= live, r.y > 0 && i + 1 >= live, r.z > 0 && i + 2 >= live, r.w > 0 && i + 3 >= live};
    int total;
    int rank = found + block_scan(f[0] + f[1] + f[2] + f[3], warp_sums, &total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) {
        source[rank] = i + k;
        place[i + k] = rank++;
      }
    found += total;
  }
  if (tid == 0) p.list[0] = found;
}

__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ PageParams p) {
  griddep_wait();
  griddep_launch_dependents();
  move_listed(p);
  const int *source = list_part(p, 0), *target = list_part(p, 1), *place = list_part(p, 2);
  const int n = p.list[0];
  if (n == 0) return;
  const size_t t = (size_t)blockIdx.x * kMoveThreads + threadIdx.x, all = (size_t)gridDim.x * kMoveThreads;
  for (size_t e = t; e < (size_t)p.D.B * p.D.max_pages; e += all) {
    const int page = p.C.page_table[e];
    if (!in_range(page, p.D.n_pages)) continue;
    const int i = place[page];
    if (in_range(i, n) && source[i] == page) p.C.page_table[e] = target[i];
  }
  for (size_t i = t; i < (size_t)n; i += all) {
    p.C.refs[target[i]] = p.C.refs[source[i]];
    p.C.refs[source[i]] = 0;
  }
}

}  // namespace paged
}  // namespace lrkv

namespace {

using namespace lrkv;
using namespace lrkv::paged;

// Arguments of a list call, and its share of the workspace.
lrkv_status list_call(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, const int32_t* src,
                      const int32_t* dst, int32_t n, void* ws, size_t ws_bytes, PageParams* p) {
  const lrkv_status st = paged::check_all(dims, cache);
  if (st != LRKV_OK) return st;
  if (n < 0) return LRKV_ERR_INVALID_ARG;
  if (n > (1 << 24)) return LRKV_ERR_UNSUPPORTED;
  if (n > 0 && (!src || !dst)) return LRKV_ERR_INVALID_ARG;
  if (!ws) return LRKV_ERR_INVALID_ARG;
  if (!aligned16(src) || !aligned16(dst) || !aligned16(ws)) return LRKV_ERR_ALIGNMENT;
  const PagedWs L = paged_ws(*dims, 1);
  if (ws_bytes < L.recs) return LRKV_ERR_INVALID_ARG;
  unsigned char* base = static_cast<unsigned char*>(ws);
  p->D = *dims;
  p->C = *cache;
  p->src = src;
  p->dst = dst;
  p->n = n;
  p->claims = reinterpret_cast<int*>(base + L.claims);
  p->ticket = reinterpret_cast<int*>(base + L.ticket);
  p->list = reinterpret_cast<int*>(base + L.list);
  p->half = dims->n_pages > dims->B ? dims->n_pages : dims->B;
  return LRKV_OK;
}

// CTAs of a kernel that moves pages: up to 64 for every SM, several waves of those that fit, not
// more than there may be work for.  Compacting 600 MB: 109 us with 8 for every SM, 99 with 64,
// 123 with 256.
unsigned move_grid(const lrkv_paged_dims& D, long long pages, long long rows) {
  const long long pieces = ((long long)page_elems(D) + kMoveBytes - 1) / kMoveBytes;
  long long n = pages * D.n_layers * pieces;
  if (n < rows) n = rows;
  const long long cap = 64LL * num_sms();
  return (unsigned)(n < 1 ? 1 : n > cap ? cap : n);
}

lrkv_status count_call(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, int32_t t_new,
                       const int32_t* t_new_b, PageParams* p) {
  const lrkv_status st = paged::check_all(dims, cache);
  if (st != LRKV_OK) return st;
  if (t_new < 0) return LRKV_ERR_INVALID_ARG;
  if (t_new > (1 << 24)) return LRKV_ERR_UNSUPPORTED;
  if (!aligned16(t_new_b)) return LRKV_ERR_ALIGNMENT;
  p->D = *dims;
  p->C = *cache;
  p->t_new_b = t_new_b;
  p->t_new = t_new;
  return LRKV_OK;
}

}  // namespace

extern "C" {

lrkv_status lrkv_pages_reserve(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, int32_t t_new,
                               const int32_t* t_new_b, void* stream) {
  PageParams p = {};
  const lrkv_status st = count_call(dims, cache, t_new, t_new_b, &p);
  if (st != LRKV_OK || t_new == 0) return st;
  return launch_pdl(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream), p);
}

lrkv_status lrkv_pages_advance(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, int32_t t_new,
                               const int32_t* t_new_b, void* stream) {
  PageParams p = {};
  const lrkv_status st = count_call(dims, cache, t_new, t_new_b, &p);
  if (st != LRKV_OK || t_new == 0) return st;
  constexpr int kWarps = kMoveThreads / 32;
  return launch_pdl(advance_kernel, dim3((unsigned)((dims->B + kWarps - 1) / kWarps)), dim3(kMoveThreads), 0,
                    static_cast<cudaStream_t>(stream), p);
}

lrkv_status lrkv_pages_fork(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, const int32_t* src,
                            const int32_t* dst, int32_t n, void* ws, size_t ws_bytes, void* stream) {
  PageParams p = {};
  lrkv_status st = list_call(dims, cache, src, dst, n, ws, ws_bytes, &p);
  if (st != LRKV_OK || n == 0) return st;
  if (n > kMaxSeqList) return LRKV_ERR_UNSUPPORTED;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p)) != LRKV_OK) return st;
  return launch_pdl(fork_move_kernel, dim3(move_grid(*dims, n, n)), dim3(kMoveThreads), 0, s, p);
}

lrkv_status lrkv_pages_free(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, const int32_t* seqs,
                            int32_t n, void* stream) {
  const lrkv_status st = paged::check_all(dims, cache);
  if (st != LRKV_OK) return st;
  if (n < 0 || (n > 0 && !seqs)) return LRKV_ERR_INVALID_ARG;
  if (n > kMaxSeqList) return LRKV_ERR_UNSUPPORTED;
  if (!aligned16(seqs)) return LRKV_ERR_ALIGNMENT;
  if (n == 0) return LRKV_OK;
  PageParams p = {};
  p.D = *dims;
  p.C = *cache;
  p.src = seqs;
  p.n = n;
  return launch_pdl(free_kernel, dim3(move_grid(*dims, 0, n)), dim3(kMoveThreads), 0,
                    static_cast<cudaStream_t>(stream), p);
}

lrkv_status lrkv_pages_copy(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, const int32_t* src,
                            const int32_t* dst, int32_t n, void* ws, size_t ws_bytes, void* stream) {
  PageParams p = {};
  lrkv_status st = list_call(dims, cache, src, dst, n, ws, ws_bytes, &p);
  if (st != LRKV_OK || n == 0) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((st = launch_pdl(copy_claim_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p)) != LRKV_OK) return st;
  return launch_pdl(copy_move_kernel, dim3(move_grid(*dims, n, 1)), dim3(kMoveThreads), 0, s, p);
}

lrkv_status lrkv_pages_compact(const lrkv_paged_dims* dims, const lrkv_paged_cache* cache, void* ws, size_t ws_bytes,
                               void* stream) {
  PageParams p = {};
  const lrkv_status st = list_call(dims, cache, nullptr, nullptr, 0, ws, ws_bytes, &p);
  if (st != LRKV_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const lrkv_status st2 = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
  if (st2 != LRKV_OK) return st2;
  return launch_pdl(compact_move_kernel, dim3(move_grid(*dims, dims->n_pages, 1)), dim3(kMoveThreads), 0, s, p);
}

}  // extern "C"
