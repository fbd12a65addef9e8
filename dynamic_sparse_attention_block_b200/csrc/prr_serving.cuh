// prr_serving.cuh -- what the calls around the decode step share: their workspace, the
// packed-row rules and the host launchers.
#pragma once

#include "prr_kernels.cuh"

namespace prr {

// Byte offsets inside the serving workspace (all 256-byte aligned).
struct ServeLayout {
  size_t status;   // int32 status word
  size_t pages;    // page bookkeeping, int32 words (see pages.cu)
  size_t attend;   // plan and partials of the attention calls (see attend.cu)
  size_t total;
};

// Rows [r0, r1) of sequence b, checked against the packed arrays.  False (and the status
// word, from the thread that passes `tell`) when the range leaves them.
__device__ __forceinline__ bool packed_range(const int* q_begin, int b, int rows, int* r0, int* r1, int* status,
                                             bool tell) {
  *r0 = q_begin[b];
  *r1 = q_begin[b + 1];
  if (*r0 >= 0 && *r0 <= *r1 && *r1 <= rows) return true;
  if (tell) report(status, kDevBadRange);
  return false;
}

constexpr int kPlanThreads = 1024;  // of the one CTA that plans a call

// Exclusive prefix sum of v over a CTA of kPlanThreads threads; *total = the sum.
template <typename T>
__device__ T cta_scan(T v, T* total) {
  __shared__ T warp_sum[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous scan's readers are done
  if (lane == 31) warp_sum[w] = x;
  __syncthreads();
  if (w == 0) {
    T s = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  *total = warp_sum[kPlanThreads / 32 - 1];
  return x - v + (w ? warp_sum[w - 1] : 0);
}

struct AppendArgs {
  const uint16_t* k_rows;
  const uint16_t* v_rows;
  long long stride;  // elements between two rows
  const int* q_begin;
  int rows;
  int* seq_lens;
  uint16_t* kc;
  uint16_t* vc;
  uint16_t* summ;
};

struct AttendArgs {
  const uint16_t* q;
  long long q_stride;
  const int* q_begin;  // packed prompts; null: a batch in groups
  int rows;
  const int* members;
  const int* group_begin;
  const int* shared_blocks;
  int n_members, n_groups;
  uint16_t* out;
  float* lse;
  void* work;    // the workspace's part for these calls, laid out for max_rows packed rows
  int max_rows;
};

constexpr int kTicketWord = 32;  // int32 word of the workspace: CTAs of a launch that are done; 0 between launches

constexpr int kMaxAttendCtas = 160;  // the workspace holds partials for so many

struct PageArgs {
  uint16_t* kc;
  uint16_t* vc;
  int* table;
  int* refs;
  int* seq_lens;
  uint16_t* summ;
  double* ema;
  int* pred;
  uint8_t* rep;
  int pred_words;   // int32 of pred per sequence
  int ema_rows;     // EMA rows of maxnb entries per sequence
  int rep_bytes;    // representative offsets per block
  int* work;        // page bookkeeping of the workspace
};

size_t page_work_words(int B, int pages);
size_t attend_tiles(int B, int max_rows, int G);
size_t attend_work_bytes(int B, int Hq, int G, int d, int max_rows);

cudaError_t launch_append_prompt(const Params& p, const AppendArgs& a, cudaStream_t s);
cudaError_t launch_attend(const Params& p, const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, int sms, cudaStream_t s);
cudaError_t launch_cache_reserve(const Params& p, const PageArgs& a, const int* want, cudaStream_t s);
cudaError_t launch_cache_fork(const Params& p, const PageArgs& a, const int* parents, const int* children, int n,
                              cudaStream_t s);
cudaError_t launch_cache_release(const Params& p, const PageArgs& a, const int* seqs, int n, cudaStream_t s);
cudaError_t launch_cache_compact(const Params& p, const PageArgs& a, int* remap, int* n_live, cudaStream_t s);

}  // namespace prr
