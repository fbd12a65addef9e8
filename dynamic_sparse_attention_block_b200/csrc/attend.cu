// attend.cu -- dense attention over the caches: packed causal prompts, and a batch in
// groups that share prefixes.
//
// Per query row q and head: s_j = scale * q . k_j over its tokens j, out = sum_j softmax(s)_j v_j,
// lse = log sum_j exp(s_j).  This is the plain kernel: one warp per (row, query head),
// 32 tokens at a time with the running maximum and sum of the softmax (one token per lane
// for q . k, d/32 channels per lane for the sum over v).
#include "prr_serving.cuh"

namespace prr {

namespace {

template <int D>
__global__ void attend_rows_kernel(const __grid_constant__ Params p, const __grid_constant__ AttendArgs a) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, hq = h * p.G + (threadIdx.x >> 5);
  const bool tell = threadIdx.x == 0 && h == 0;
  int seq, first, shared_to = 0, row, n;  // tokens [0, n); below shared_to through `first`
  if (a.q_begin) {
    row = blockIdx.x;
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.q_begin[mid] <= row) lo = mid;
      else hi = mid - 1;
    }
    first = seq = lo;
    int r0, r1;
    if (!packed_range(a.q_begin, seq, a.rows, &r0, &r1, p.status, tell) || row < r0 || row >= r1) return;
    const int len = p.seq_lens[seq];
    if (len < 1 || len > p.cap || r1 - r0 > len) {
      if (tell) report(p.status, kDevBadSeqLen);
      return;
    }
    n = len - (r1 - r0) + (row - r0) + 1;
  } else {
    const int i = blockIdx.x;
    int lo = 0, hi = a.n_groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.group_begin[mid] <= i) lo = mid;
      else hi = mid - 1;
    }
    const int g0 = a.group_begin[lo], g1 = a.group_begin[lo + 1], sb = a.shared_blocks[lo];
    if (g0 < 0 || g0 > i || g1 <= i || g1 > a.n_members || sb < 0 || sb > p.maxnb) {
      if (tell && g1 != g0) report(p.status, kDevBadRange);
      return;
    }
    seq = row = a.members[i];
    first = a.members[g0];
    if (seq < 0 || seq >= p.B || first < 0 || first >= p.B) {
      if (tell) report(p.status, kDevBadRange);
      return;
    }
    n = p.seq_lens[seq];
    if (n < 0 || n > p.cap) {
      if (tell) report(p.status, kDevBadSeqLen);
      return;
    }
    shared_to = sb * p.bs;
    if (shared_to > n) {
      if (tell) report(p.status, kDevBadRange);
      return;
    }
  }

  constexpr int C = D / 32;  // channels per lane
  const uint16_t* q = a.q + static_cast<size_t>(row) * a.q_stride + static_cast<size_t>(hq) * D;
  float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
  for (int i = 0; i < C; ++i) o[i] = 0.f;
  for (int t0 = 0; t0 < n; t0 += 32) {  // a tile of 32 tokens lies in one block
    const long long r = kv_row(p, (t0 < shared_to ? first : seq) * p.Hkv + h, t0);
    if (r < 0) continue;
    float s = -INFINITY;
    if (t0 + lane < n) {
      const uint4* kr = reinterpret_cast<const uint4*>(p.kc + static_cast<size_t>(r + lane) * D);
      s = 0.f;
      for (int c = 0; c < D / 8; ++c) {
        const uint4 kw = kr[c], qw = reinterpret_cast<const uint4*>(q)[c];
        const uint32_t kk[4] = {kw.x, kw.y, kw.z, kw.w}, qq[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) s += bf16_lo(kk[e]) * bf16_lo(qq[e]) + bf16_hi(kk[e]) * bf16_hi(qq[e]);
      }
      s *= p.scale_log2;
    }
    float mt = s;
#pragma unroll
    for (int x = 16; x; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, x));
    const float mn = fmaxf(m, mt), base = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - base), w = exp2f(s - base);
    float ws = w;
#pragma unroll
    for (int x = 16; x; x >>= 1) ws += __shfl_xor_sync(0xFFFFFFFFu, ws, x);
    l = l * f + ws;
    m = mn;
#pragma unroll
    for (int i = 0; i < C; ++i) o[i] *= f;
    for (int t = 0; t < min(32, n - t0); ++t) {
      const float wt = __shfl_sync(0xFFFFFFFFu, w, t);
      const uint16_t* vr = p.vc + static_cast<size_t>(r + t) * D + lane * C;
#pragma unroll
      for (int i = 0; i < C; ++i) o[i] += wt * __uint_as_float(static_cast<uint32_t>(vr[i]) << 16);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t at = static_cast<size_t>(row) * p.Hq + hq;
#pragma unroll
  for (int i = 0; i < C; ++i) reinterpret_cast<__nv_bfloat16*>(a.out)[at * D + lane * C + i] = __float2bfloat16(o[i] * inv);
  if (a.lse && lane == 0) a.lse[at] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

cudaError_t launch_attend(const Params& p, const AttendArgs& a, cudaStream_t s) {
  const dim3 grid(a.q_begin ? a.rows : a.n_members, p.Hkv), block(32 * p.G);
  return p.d == 128 ? launch_kernel(attend_rows_kernel<128>, grid, block, 0, s, 0, p, a)
                    : launch_kernel(attend_rows_kernel<64>, grid, block, 0, s, 0, p, a);
}

}  // namespace prr
