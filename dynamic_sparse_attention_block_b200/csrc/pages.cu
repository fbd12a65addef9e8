// pages.cu -- the pages of a paged cache: reserving, forking, releasing, compacting.
//
// The state is the block table and one reference count per page; a page is free at 0 (or below).
// Free pages are always given out lowest first, in the order of the requests, so the
// tables do not depend on the order in which threads run.  The plans (which page goes
// where) are integer scans over the counts by one CTA, a launch that the copies wait for; the
// copies are bound by HBM.  Measured (B200): 60 forks of 128K sequences (summaries, state and last pages, 511 MB)
// with their release and reservation in 99 us, 5.1 TB/s; 2048 moved pages of 512 KB in 440 us, 4.9 TB/s (75% of a
// measured copy).
#include "prr_serving.cuh"

namespace prr {

namespace {

constexpr int kPlanEach = 8;  // neighbouring pages a thread looks at between two scans

// Page bookkeeping in the workspace, int32 words.
struct PageWork {
  int* list;    // [pages] free pages in ascending order; compaction: the holes below L
  int* movers;  // [pages] compaction: live pages at L and above, ascending
  int* need;    // [B] pages the request wants; then its first rank
  int* claim;   // [B] fork: the first entry that names a child
  int* src;     // [B] fork: page copied from (-1: none)
  int* dst;     // [B] fork: page copied to
  int* len;     // [B] fork: the parent's length (-1: this entry is skipped)
  int* count;   // [4] compaction: moves
};

__host__ __device__ inline PageWork page_work(int* w, int B, int pages) {
  PageWork x;
  x.list = w;
  x.movers = x.list + pages;
  x.need = x.movers + pages;
  x.claim = x.need + B;
  x.src = x.claim + B;
  x.dst = x.src + B;
  x.len = x.dst + B;
  x.count = x.len + B;
  return x;
}

// The `need` lowest free pages, ascending, into list.  Returns how many there are (need,
// or fewer).
__device__ int find_free(const int* refs, int pages, int need, int* list) {
  int found = 0;
  for (long long base = 0; base < pages && found < need; base += kPlanThreads * kPlanEach) {
    const long long i0 = base + threadIdx.x * kPlanEach;
    unsigned free_pages = 0;
#pragma unroll
    for (int u = 0; u < kPlanEach; ++u)
      if (i0 + u < pages && refs[i0 + u] <= 0) free_pages |= 1u << u;
    int total;
    int at = found + cta_scan(__popc(free_pages), &total);
    for (; free_pages && at < need; free_pages &= free_pages - 1) list[at++] = static_cast<int>(i0) + __ffs(free_pages) - 1;
    found = min(need, found + total);
  }
  __syncthreads();
  return found;
}

// Exclusive prefix sums over need[0..n) in place; returns the sum, which may pass 32 bits (a table can have more
// entries; the sums in place then mean nothing).
__device__ long long scan_needs(int* need, int n) {
  long long sum = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    long long total;
    const long long at = sum + cta_scan<long long>(i < n ? need[i] : 0, &total);
    if (i < n) need[i] = static_cast<int>(at);
    sum += total;
  }
  __syncthreads();
  return sum;
}

// Blocks of sequence b that a reservation looks at: [lo, hi).
__device__ void wanted(const Params& p, const PageArgs& a, const int* want, int b, int* lo, int* hi, bool tell) {
  const int len = a.seq_lens[b], w = want[b];
  *lo = *hi = 0;
  if (w <= 0) return;
  if (w > p.cap || len < 0 || len > p.cap) {
    if (tell) report(p.status, kDevBadSeqLen);
    return;
  }
  *lo = (len + p.bs - 1) / p.bs;
  *hi = (w + p.bs - 1) / p.bs;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const __grid_constant__ Params p,
                                                               const __grid_constant__ PageArgs a, const int* want) {
  const PageWork w = page_work(a.work, p.B, p.pages);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int b = warp; b < p.B; b += kPlanThreads / 32) {
    int lo, hi, n = 0;
    wanted(p, a, want, b, &lo, &hi, lane == 0);
    for (int j = lo + lane; j < hi; j += 32) n += a.table[static_cast<size_t>(b) * p.maxnb + j] < 0;
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) w.need[b] = n;
  }
  __syncthreads();
  const long long need = scan_needs(w.need, p.B);
  if (need == 0) return;
  if (need > p.pages || find_free(a.refs, p.pages, static_cast<int>(need), w.list) < need) {
    if (threadIdx.x == 0) report(p.status, kDevNoPages);
    return;
  }
  for (int b = warp; b < p.B; b += kPlanThreads / 32) {
    int lo, hi, at = w.need[b];
    wanted(p, a, want, b, &lo, &hi, false);
    for (int j0 = lo; j0 < hi; j0 += 32) {
      const int j = j0 + lane;
      int* e = a.table + static_cast<size_t>(b) * p.maxnb + j;
      const bool miss = j < hi && *e < 0;
      const unsigned m = __ballot_sync(0xFFFFFFFFu, miss);
      if (miss) {
        const int pg = w.list[at + __popc(m & ((1u << lane) - 1))];
        *e = pg;
        a.refs[pg] = 1;
      }
      at += __popc(m);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const __grid_constant__ Params p,
                                                                 const __grid_constant__ PageArgs a,
                                                                 const int* parents, const int* children, int n) {
  const PageWork w = page_work(a.work, p.B, p.pages);
  for (int b = threadIdx.x; b < p.B; b += kPlanThreads) w.claim[b] = n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int c = children[i];
    if (c >= 0 && c < p.B) atomicMin(&w.claim[c], i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int c = children[i], f = parents[i];
    int len = -1, src = -1;
    if (c < 0 || c >= p.B || f < 0 || f >= p.B || w.claim[c] != i || w.claim[f] != n || a.seq_lens[c] != 0 ||
        a.table[static_cast<size_t>(c) * p.maxnb] >= 0) {
      report(p.status, kDevBadRange);
    } else {
      len = a.seq_lens[f];
      if (len < 0 || len > p.cap) {
        report(p.status, kDevBadSeqLen);
        len = -1;
      } else if (len % p.bs) {
        src = a.table[static_cast<size_t>(f) * p.maxnb + len / p.bs];
        if (src < 0 || src >= p.pages) {
          report(p.status, kDevBadRange);
          src = len = -1;
        }
      }
    }
    w.src[i] = src;
    w.len[i] = len;
    w.need[i] = src >= 0;
  }
  __syncthreads();
  const int need = static_cast<int>(scan_needs(w.need, n));  // at most n
  const bool enough = need == 0 || find_free(a.refs, p.pages, need, w.list) == need;
  if (!enough && threadIdx.x == 0) report(p.status, kDevNoPages);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    if (!enough) w.len[i] = -1;
    w.dst[i] = enough && w.src[i] >= 0 ? w.list[w.need[i]] : -1;
  }
}

// Bulk copy by a whole CTA; both pointers 16-byte aligned, bytes a multiple of 16.
__device__ void copy16(void* dst, const void* src, size_t bytes, int part, int parts) {
  const uint4* s = static_cast<const uint4*>(src);
  uint4* d = static_cast<uint4*>(dst);
  const size_t n = bytes / 16, step = static_cast<size_t>(parts) * blockDim.x;
#pragma unroll 4
  for (size_t i = static_cast<size_t>(part) * blockDim.x + threadIdx.x; i < n; i += step) d[i] = s[i];
}

// CTAs per child.  With 8, 32, 128: one child of 131K tokens 90, 39, 27 us; 60 of them 121, 94, 94; 60 children of 2K tokens
// 39, 40, 61; one of 1K 33, 27, 25.
constexpr int kForkParts = 32;

__global__ void __launch_bounds__(256) fork_copy_kernel(const __grid_constant__ Params p,
                                                        const __grid_constant__ PageArgs a, const int* parents,
                                                        const int* children) {
  const PageWork w = page_work(a.work, p.B, p.pages);
  const int i = blockIdx.y, part = blockIdx.x;
  const int len = w.len[i];
  if (len < 0) return;
  const int f = parents[i], c = children[i];
  const int full = len / p.bs, nb = (len + p.bs - 1) / p.bs;
  const int* from = a.table + static_cast<size_t>(f) * p.maxnb;
  int* to = a.table + static_cast<size_t>(c) * p.maxnb;
  for (int j = part * blockDim.x + threadIdx.x; j < full; j += kForkParts * blockDim.x) {
    const int pg = from[j];
    to[j] = pg;
    if (pg >= 0 && pg < p.pages) atomicAdd(&a.refs[pg], 1);
    else report(p.status, kDevBadRange);
  }
  const int dst = w.dst[i];
  if (part == 0 && threadIdx.x == 0) {
    a.seq_lens[c] = len;
    if (dst >= 0) {
      to[full] = dst;
      a.refs[dst] = 1;
    }
  }
  if (dst >= 0) {
    const size_t page = static_cast<size_t>(p.Hkv) * p.bs * p.d;
    copy16(a.kc + dst * page, a.kc + w.src[i] * page, page * 2, part, kForkParts);
    copy16(a.vc + dst * page, a.vc + w.src[i] * page, page * 2, part, kForkParts);
  }
  if (a.summ) {
    const size_t row = static_cast<size_t>(p.maxnb) * 2 * p.d;
    for (int h = 0; h < p.Hkv; ++h)
      copy16(a.summ + (static_cast<size_t>(c) * p.Hkv + h) * row, a.summ + (static_cast<size_t>(f) * p.Hkv + h) * row,
             static_cast<size_t>(nb) * 4 * p.d, part, kForkParts);
  }
  if (a.ema) {
    const size_t row = static_cast<size_t>(a.ema_rows) * p.maxnb;
    for (size_t e = static_cast<size_t>(part) * blockDim.x + threadIdx.x; e < row;
         e += static_cast<size_t>(kForkParts) * blockDim.x)
      a.ema[c * row + e] = e % p.maxnb < static_cast<size_t>(nb) ? a.ema[f * row + e] : 0.0;
  }
  if (a.pred && part == 0)
    for (int e = threadIdx.x; e < a.pred_words; e += blockDim.x)
      a.pred[static_cast<size_t>(c) * a.pred_words + e] = a.pred[static_cast<size_t>(f) * a.pred_words + e];
  if (a.rep) {
    const size_t row = static_cast<size_t>(p.maxnb) * a.rep_bytes, used = static_cast<size_t>(nb) * a.rep_bytes;
    for (int h = 0; h < p.Hkv; ++h)
      for (size_t e = static_cast<size_t>(part) * blockDim.x + threadIdx.x; e < used;
           e += static_cast<size_t>(kForkParts) * blockDim.x)
        a.rep[(static_cast<size_t>(c) * p.Hkv + h) * row + e] = a.rep[(static_cast<size_t>(f) * p.Hkv + h) * row + e];
  }
}

__global__ void __launch_bounds__(256) release_kernel(const __grid_constant__ Params p,
                                                      const __grid_constant__ PageArgs a, const int* seqs) {
  const int b = seqs[blockIdx.y];
  if (b < 0 || b >= p.B) {
    if (threadIdx.x == 0 && blockIdx.x == 0) report(p.status, kDevBadRange);
    return;
  }
  const int t0 = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  if (t0 == 0) a.seq_lens[b] = 0;
  if (a.ema) {
    const size_t n = static_cast<size_t>(a.ema_rows) * p.maxnb;
    for (size_t e = t0; e < n; e += step) a.ema[b * n + e] = 0.0;
  }
  if (a.pred)  // what the zero state predicts
    for (int e = t0; e < a.pred_words; e += step) a.pred[static_cast<size_t>(b) * a.pred_words + e] = e % p.P;
  int* row = a.table + static_cast<size_t>(b) * p.maxnb;
  for (int j = t0; j < p.maxnb; j += step) {
    if (row[j] == -1) continue;
    const int pg = atomicExch(&row[j], -1);  // two entries for one sequence: one of them gets the page
    if (pg == -1) continue;
    if (pg < 0 || pg >= p.pages) {
      report(p.status, kDevBadRange);
    } else if (atomicSub(&a.refs[pg], 1) <= 0) {  // a count that did not know of this row
      atomicAdd(&a.refs[pg], 1);
      report(p.status, kDevBadRange);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const __grid_constant__ Params p,
                                                                    const __grid_constant__ PageArgs a, int* remap,
                                                                    int* n_live) {
  const PageWork w = page_work(a.work, p.B, p.pages);
  int live = 0;
  for (int i = threadIdx.x; i < p.pages; i += kPlanThreads) live += a.refs[i] > 0;
  int L;
  cta_scan(live, &L);
  const int holes = find_free(a.refs, L, L, w.list);  // free pages below L
  int moves = 0;
  for (long long base = 0; base < p.pages; base += kPlanThreads * kPlanEach) {
    const long long i0 = base + threadIdx.x * kPlanEach;
    unsigned used = 0;
#pragma unroll
    for (int u = 0; u < kPlanEach; ++u)
      if (i0 + u < p.pages && a.refs[i0 + u] > 0) used |= 1u << u;
    const int below = static_cast<int>(min(max(L - i0, 0ll), static_cast<long long>(kPlanEach)));  // pages that stay
    int total;
    int at = moves + cta_scan(__popc(used >> below), &total);
    for (int u = 0; u < kPlanEach && i0 + u < p.pages; ++u) {
      const int i = static_cast<int>(i0) + u;
      if (!((used >> u) & 1)) {
        remap[i] = -1;
      } else if (u < below) {
        remap[i] = i;
      } else {
        w.movers[at] = i;
        remap[i] = w.list[at++];
      }
    }
    moves += total;
  }
  if (threadIdx.x == 0) {
    *n_live = L;
    w.count[0] = min(moves, holes);
  }
}

// Part `part` of kPageParts equal parts of a page's K or V, by one CTA: pages in parts, so that the CTAs end together
// (2048 pages of 512 KB: 451 us with whole pages, 1.7 to a CTA, 440 in parts).
constexpr int kPageParts = 8;

__device__ void copy_part(uint16_t* dst, const uint16_t* src, size_t bytes, int part) {
  const size_t n = bytes / 16 / kPageParts;  // a page is a multiple of 64 * 64 * 2 bytes
  const uint4* s = reinterpret_cast<const uint4*>(src) + part * n;
  uint4* d = reinterpret_cast<uint4*>(dst) + part * n;
#pragma unroll 8
  for (size_t i = threadIdx.x; i < n; i += blockDim.x) __stcs(d + i, __ldcs(s + i));
}

// Eight CTAs an SM copy (592, 1184, 2368 of them: 2048 pages of 512 KB 444, 438, 434 us, 150 of 256 small pages 14, 14, 16);
// the table's number does not show (37 or 148).
constexpr int kCompactCopyCtas = 1184, kCompactTableCtas = 148;

// The pages that move, and in the last CTAs the table entries and counts that follow them.
__global__ void __launch_bounds__(256) compact_move_kernel(const __grid_constant__ Params p,
                                                           const __grid_constant__ PageArgs a, const int* remap) {
  const PageWork w = page_work(a.work, p.B, p.pages);
  const int moves = w.count[0];
  if (blockIdx.x < kCompactCopyCtas) {
    const size_t page = static_cast<size_t>(p.Hkv) * p.bs * p.d;
    const long long items = static_cast<long long>(moves) * kPageParts;
    for (long long i = blockIdx.x; i < items; i += kCompactCopyCtas) {
      const int src = w.movers[i / kPageParts], dst = w.list[i / kPageParts], part = static_cast<int>(i % kPageParts);
      copy_part(a.kc + dst * page, a.kc + src * page, page * 2, part);
      copy_part(a.vc + dst * page, a.vc + src * page, page * 2, part);
    }
    return;
  }
  const size_t n = static_cast<size_t>(p.B) * p.maxnb, step = static_cast<size_t>(kCompactTableCtas) * blockDim.x;
  const size_t t0 = static_cast<size_t>(blockIdx.x - kCompactCopyCtas) * blockDim.x + threadIdx.x;
  for (size_t i = t0; i < n; i += step) {
    const int pg = a.table[i];
    if (pg >= 0 && pg < p.pages && remap[pg] >= 0) a.table[i] = remap[pg];
    else if (pg != -1) report(p.status, kDevBadRange);
  }
  for (size_t i = t0; i < static_cast<size_t>(moves); i += step) {
    const int src = w.movers[i], dst = w.list[i];
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
  }
}

}  // namespace

size_t page_work_words(int B, int pages) { return 2 * static_cast<size_t>(pages) + 5 * static_cast<size_t>(B) + 4; }

cudaError_t launch_cache_reserve(const Params& p, const PageArgs& a, const int* want, cudaStream_t s) {
  return launch_kernel(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, s, 0, p, a, want);
}

cudaError_t launch_cache_fork(const Params& p, const PageArgs& a, const int* parents, const int* children, int n,
                              cudaStream_t s) {
  const cudaError_t e =
      launch_kernel(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, 0, p, a, parents, children, n);
  if (e != cudaSuccess) return e;
  return launch_kernel(fork_copy_kernel, dim3(kForkParts, n), dim3(256), 0, s, 0, p, a, parents, children);
}

cudaError_t launch_cache_release(const Params& p, const PageArgs& a, const int* seqs, int n, cudaStream_t s) {
  const int parts = min(32, (p.maxnb + 255) / 256);
  return launch_kernel(release_kernel, dim3(parts, n), dim3(256), 0, s, 0, p, a, seqs);
}

cudaError_t launch_cache_compact(const Params& p, const PageArgs& a, int* remap, int* n_live, cudaStream_t s) {
  cudaError_t e = launch_kernel(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, 0, p, a, remap, n_live);
  if (e == cudaSuccess)
    e = launch_kernel(compact_move_kernel, dim3(kCompactCopyCtas + kCompactTableCtas), dim3(256), 0, s, 0, p, a,
                      static_cast<const int*>(remap));
  return e;
}

}  // namespace prr
