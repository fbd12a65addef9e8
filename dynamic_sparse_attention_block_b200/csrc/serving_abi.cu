// serving_abi.cu -- host side of the calls around the decode step: argument and shape
// rules, the serving workspace, launches.
#include <cstring>

#include "prr_host.cuh"
#include "prr_serving.cuh"

using namespace prr;

namespace {

ServeLayout serve_layout(const prr_dims* d, int32_t max_rows) {
  ServeLayout L = {};
  size_t off = 256;  // status word, and behind it (kTicketWord) a ticket
  L.pages = off;
  off = align256(off + 4 * page_work_words(d->B, d->pages));
  L.attend = off;
  off = align256(off + attend_work_bytes(d->B, d->Hq, d->Hq / d->Hkv, d->d, max_rows));
  L.total = off;
  return L;
}

bool rows_ok(int32_t rows) { return rows >= 0 && rows <= (1 << 30); }

// Distance of two packed rows of `heads` heads.
bool stride_ok(int64_t stride, int64_t heads, int64_t d) { return stride >= heads * d && stride % 8 == 0; }

// Tensor maps of the caches and the launch, for both attention calls.
prr_status attend(const prr_dims* d, Params& p, AttendArgs& a, void* ws, const ServeLayout& L, int32_t max_rows,
                  cudaStream_t stream) {
  a.work = static_cast<unsigned char*>(ws) + L.attend;
  a.max_rows = max_rows;
  CUtensorMap qm = {}, km, vm;
  if (!make_kv_step_map(&km, p.kc, d) || !make_kv_step_map(&vm, p.vc, d)) return PRR_ERR_CUDA;
  if (a.q_begin && !make_q_map(&qm, a.q, a.q_stride, a.rows, d)) return PRR_ERR_CUDA;
  return cuda_status(launch_attend(p, a, qm, km, vm, device_info().sms, stream));
}

// The kernel parameters that these calls read.
Params serve_params(const prr_dims* d, void* ws, const ServeLayout& L) {
  Params p;
  std::memset(&p, 0, sizeof p);
  p.B = d->B;
  p.Hq = d->Hq;
  p.Hkv = d->Hkv;
  p.G = d->Hq / d->Hkv;
  p.upb = d->Hkv;
  p.kv_div = 1;
  p.units = d->B * d->Hkv;
  p.d = d->d;
  p.bs = d->bs;
  p.cap = d->cap_tokens;
  p.K = d->K;
  p.P = d->P;
  p.maxnb = (d->cap_tokens + d->bs - 1) / d->bs;
  p.pages = d->pages;
  p.table = d->block_table;
  p.scale_log2 = static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634074);
  p.status = reinterpret_cast<int*>(static_cast<unsigned char*>(ws) + L.status);
  return p;
}

// The buffers every prr_cache_* call needs, and the kernels' view of them.
prr_status page_args(const prr_dims* d, const prr_cache_buffers* c, void* ws, size_t ws_bytes, Params* p, PageArgs* a) {
  if (!dims_ok(d) || d->pages == 0) return PRR_ERR_SHAPE;
  if (!c || !ws || !c->block_table || !c->page_refs) return PRR_ERR_INVALID_ARG;
  if (c->block_table != d->block_table) return PRR_ERR_INVALID_ARG;
  if ((c->k_cache && !aligned16(c->k_cache)) || (c->v_cache && !aligned16(c->v_cache)) || (c->summ && !aligned16(c->summ)))
    return PRR_ERR_INVALID_ARG;
  const ServeLayout L = serve_layout(d, 1);
  if (ws_bytes < L.total) return PRR_ERR_CAPACITY;
  *p = serve_params(d, ws, L);
  const int per_seq = d->selector == PRR_SELECT_PER_HEAD ? d->Hq : d->Hkv;
  a->kc = c->k_cache;
  a->vc = c->v_cache;
  a->table = c->block_table;
  a->refs = c->page_refs;
  a->seq_lens = c->seq_lens;
  a->summ = c->summ;
  a->ema = c->ema;
  a->pred = d->P > 0 ? c->pred : nullptr;
  a->rep = d->selector == PRR_SELECT_REPRESENTATIVE ? c->rep_offsets : nullptr;
  a->pred_words = per_seq * d->P;
  a->ema_rows = per_seq;
  a->rep_bytes = d->n_rep;
  a->work = reinterpret_cast<int*>(static_cast<unsigned char*>(ws) + L.pages);
  return PRR_OK;
}

}  // namespace

extern "C" {

size_t prr_serving_workspace_bytes(const prr_dims* dims, int32_t max_rows) {
  if (!dims_ok(dims) || max_rows < 1 || !rows_ok(max_rows)) return 0;
  return serve_layout(dims, max_rows).total;
}

prr_status prr_append_prompt(const prr_dims* dims, const uint16_t* k_rows, const uint16_t* v_rows, int64_t row_stride,
                             const int32_t* q_begin, int32_t rows, int32_t* seq_lens, uint16_t* k_cache,
                             uint16_t* v_cache, uint16_t* summ, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!dims_ok(dims) || !rows_ok(rows) || !stride_ok(row_stride, dims->Hkv, dims->d)) return PRR_ERR_SHAPE;
  if (rows == 0) return PRR_OK;
  if (!k_rows || !v_rows || !q_begin || !seq_lens || !k_cache || !v_cache || !ws) return PRR_ERR_INVALID_ARG;
  if (!aligned16(k_rows) || !aligned16(v_rows) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(summ))
    return PRR_ERR_INVALID_ARG;
  const ServeLayout L = serve_layout(dims, 1);
  if (ws_bytes < L.total) return PRR_ERR_CAPACITY;
  const Params p = serve_params(dims, ws, L);
  const AppendArgs a = {k_rows, v_rows, row_stride, q_begin, rows, seq_lens, k_cache, v_cache, summ};
  return cuda_status(launch_append_prompt(p, a, stream));
}

prr_status prr_attend_prompt(const prr_dims* dims, const uint16_t* q, int64_t q_stride, const int32_t* q_begin,
                             int32_t rows, const int32_t* seq_lens, const uint16_t* k_cache, const uint16_t* v_cache,
                             uint16_t* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  if (!dims_ok(dims) || !rows_ok(rows) || !stride_ok(q_stride, dims->Hq, dims->d)) return PRR_ERR_SHAPE;
  if (rows == 0) return PRR_OK;
  if (!q || !q_begin || !seq_lens || !k_cache || !v_cache || !out || !ws) return PRR_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PRR_ERR_INVALID_ARG;
  const ServeLayout L = serve_layout(dims, rows);
  if (ws_bytes < L.total) return PRR_ERR_CAPACITY;
  Params p = serve_params(dims, ws, L);
  p.kc = k_cache;
  p.vc = v_cache;
  p.seq_lens = seq_lens;
  AttendArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.q_begin = q_begin;
  a.rows = rows;
  a.out = out;
  a.lse = lse;
  return attend(dims, p, a, ws, L, rows, stream);
}

prr_status prr_attend_shared(const prr_dims* dims, const uint16_t* q, int64_t q_stride, const int32_t* members,
                             int32_t n_members, const int32_t* group_begin, const int32_t* shared_blocks,
                             int32_t n_groups, const int32_t* seq_lens, const uint16_t* k_cache,
                             const uint16_t* v_cache, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                             cudaStream_t stream) {
  if (!dims_ok(dims) || !stride_ok(q_stride, dims->Hq, dims->d)) return PRR_ERR_SHAPE;
  if (n_members < 0 || n_members > dims->B || n_groups < 0 || n_groups > dims->B) return PRR_ERR_SHAPE;
  if (n_groups == 0 || n_members == 0) return PRR_OK;
  if (!q || !members || !group_begin || !shared_blocks || !seq_lens || !k_cache || !v_cache || !out || !ws)
    return PRR_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PRR_ERR_INVALID_ARG;
  const ServeLayout L = serve_layout(dims, 1);
  if (ws_bytes < L.total) return PRR_ERR_CAPACITY;
  Params p = serve_params(dims, ws, L);
  p.kc = k_cache;
  p.vc = v_cache;
  p.seq_lens = seq_lens;
  AttendArgs a = {};
  a.q = q;
  a.q_stride = q_stride;
  a.members = members;
  a.group_begin = group_begin;
  a.shared_blocks = shared_blocks;
  a.n_members = n_members;
  a.n_groups = n_groups;
  a.out = out;
  a.lse = lse;
  return attend(dims, p, a, ws, L, 1, stream);
}

prr_status prr_cache_reserve(const prr_dims* dims, const int32_t* want_lens, const prr_cache_buffers* cache, void* ws,
                             size_t ws_bytes, cudaStream_t stream) {
  Params p;
  PageArgs a;
  const prr_status st = page_args(dims, cache, ws, ws_bytes, &p, &a);
  if (st != PRR_OK) return st;
  if (!want_lens || !a.seq_lens) return PRR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_reserve(p, a, want_lens, stream));
}

prr_status prr_cache_fork(const prr_dims* dims, const int32_t* parents, const int32_t* children, int32_t n,
                          const prr_cache_buffers* cache, void* ws, size_t ws_bytes, cudaStream_t stream) {
  Params p;
  PageArgs a;
  const prr_status st = page_args(dims, cache, ws, ws_bytes, &p, &a);
  if (st != PRR_OK) return st;
  if (n < 0 || n > dims->B) return PRR_ERR_SHAPE;
  if (n == 0) return PRR_OK;
  if (!parents || !children || !a.seq_lens || !a.kc || !a.vc) return PRR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_fork(p, a, parents, children, n, stream));
}

prr_status prr_cache_release(const prr_dims* dims, const int32_t* seqs, int32_t n, const prr_cache_buffers* cache,
                             void* ws, size_t ws_bytes, cudaStream_t stream) {
  Params p;
  PageArgs a;
  const prr_status st = page_args(dims, cache, ws, ws_bytes, &p, &a);
  if (st != PRR_OK) return st;
  if (n < 0 || n > dims->B) return PRR_ERR_SHAPE;
  if (n == 0) return PRR_OK;
  if (!seqs || !a.seq_lens) return PRR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_release(p, a, seqs, n, stream));
}

prr_status prr_cache_compact(const prr_dims* dims, const prr_cache_buffers* cache, int32_t* remap, int32_t* n_live,
                             void* ws, size_t ws_bytes, cudaStream_t stream) {
  Params p;
  PageArgs a;
  const prr_status st = page_args(dims, cache, ws, ws_bytes, &p, &a);
  if (st != PRR_OK) return st;
  if (!remap || !n_live || !a.kc || !a.vc) return PRR_ERR_INVALID_ARG;
  return cuda_status(launch_cache_compact(p, a, remap, n_live, stream));
}

}  // extern "C"
