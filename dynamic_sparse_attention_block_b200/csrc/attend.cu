// attend.cu -- dense attention over the caches: packed causal prompts, and a batch in
// groups that share prefixes.
//
// Per query row and head: s_j = scale * q . k_j over its tokens j,
//   out = sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m),   lse = (m + log2 sum) ln 2,   s' = s log2 e,
// in one pass over the tokens with a running reference m (tensor cores for both products).
//
// Tiles.  A tile is up to 256 rows that read the same tokens of one KV head: the G query
// heads of its group times up to 2 * floor(128/G) packed tokens of one prompt, or the G heads of
// that many members of a group (over the shared prefix) or of one sequence (over its own
// tokens).  Its work is counted in blocks of 128 tokens.  The plan kernel numbers all (head, tile,
// block) units and cuts them into equal runs, one per CTA, wherever the cuts fall -- so prompts,
// single tokens, long prefixes and ragged batches all fill the machine evenly.  A tile cut
// between CTAs (and every tile of a batch in groups) leaves fp32 partials (m, sum, O) that the
// combine kernels merge.
//
// A CTA (one per SM) works on a piece of a tile, in steps of 64 tokens:
//  - one thread per half (128 rows) issues its products on the tensor cores: S = Q K^T into tensor
//    memory, O += P V with P read from there.  S is asked for one step ahead (two buffers of 64
//    columns; with O, 2 x d columns, tensor memory is full);
//  - a warp copies K and V by TMA into a ring of stages, another brings the next piece's Q;
//  - two groups of 128 threads, one thread to a row, turn S into P = 2^(s' - m) in place.
// A tile of up to 128 rows is split: both halves take its rows, each every other step, and merge
// through tensor memory at the end.
//
// P is rounded to bf16 (the products' operand type): half a step, 2^-8 of each weight at most;
// its sum, m and O stay fp32, and the result is rounded once.  m only moves when a row's
// maximum grew by more than 2^8: until then weights up to 256 stay in range, and O needs no rescaling.
//
// A maximum passes over NaN, a sum does not: partials of no token are told by sum = 0, and a row of scores that are
// not finite carries its NaN through every merge (m is -infinity for both).
//
// Measured (B200, 32/8 heads, d 128): a 32K prompt in 8.3 to 8.6 ms, 1020 to 1060 TFLOP/s or 62 to 64%
// of a measured matrix product; bound by the softmax's latency and the products (tensor pipe 75% busy; Q K^T with
// 64 columns is limited by shared memory, 48 clocks where 128 columns take 64).  One step of 128 tokens
// without S ahead: 900 TFLOP/s.  64 queries of 64/8 heads on four prefixes of 128K: 490 to 520 us,
// 4.3 to 4.6 TB/s or 66 to 70% of a measured copy; the prefixes alone in 370 to 420 us.  Pieces of 1024 rows of two
// prompts behind 63K tokens (64/8 heads, caches of 0.53 GB): 920 to 1010 TFLOP/s, with 15.8 GB read from DRAM, as the CTAs
// of a head stand at unrelated tokens; the same work on caches that stay in L2 (37 MB) 1240.
#include "prr_serving.cuh"
#include "prr_tensor.cuh"

namespace prr {

namespace {

constexpr int kBlock = 128;         // tokens per unit of work
constexpr int kStep = 64;           // tokens per product: two steps of S in tensor memory, one ahead
constexpr float kGrow = 8.0f;       // log2 of the growth that moves the reference m
constexpr int kAttendThreads = 384;  // 2 x 128 softmax threads; two warps for products, one for copies, one for Q

__host__ __device__ constexpr int sub_tokens(int G) { return kBlock / G; }  // packed tokens per 128 rows

struct Tile {  // 32 bytes
  int row0;    // first entry of the row list
  int ntok;    // packed tokens (each G rows)
  int seq;     // whose tokens it reads
  int kv0;     // first token
  int kv1;     // one past the last
  int pos0;    // causal: position of the first packed token; kNoMask: every row reads all of [kv0, kv1)
  int blocks;  // weight
  int part0;   // first row of its partials (batch in groups)
};
constexpr int kNoMask = 1 << 30;

struct Start {  // a CTA's run: where it begins, how long it is, and its first tile
  int head, tile, off, count;  // count: tiles of the plan
  long long left;
  int pieces;  // of that tile, where this is the first cut through it: its pieces are of CTAs c - 1, c, ...; else 0
  int pad;
  Tile first;
};

struct PlanHead {
  long long per_head;  // units of one KV head
  int tiles;
  int ctas;            // CTAs with work
};

struct Plan {
  PlanHead* head;
  Start* start;        // [kMaxAttendCtas]
  long long* prefix;   // [tiles + 1] units before each tile
  Tile* tile;
  int* row;            // [B] batch in groups: the sequence of each entry, -1: skipped
  float* part;         // partial rows: m, sum, O[d]
};

__host__ __device__ inline long long first_unit(long long units, int ctas, int c) { return units * c / ctas; }
// The CTA whose run has unit z: the last with first_unit <= z.
__device__ __forceinline__ int cta_of(long long units, int ctas, long long z) {
  return static_cast<int>(((z + 1) * ctas - 1) / units);
}

// ------------------------------------------------------------------ the plan

// The plan's small inputs and its prefix sums are searched in shared memory where they fit.
constexpr int kPlanSeqs = 2048, kPlanSlots = 2048;

// Tile `slot` of packed prompts.  Sequence b owns the slots floor(q_begin[b] / span) + b
// ...: at least as many as it has tiles, so a slot finds its tile by bisection; slots left over weigh 0.
__device__ Tile prompt_tile(const Params& p, const AttendArgs& a, const int* q_begin, int slot, int span) {
  Tile t = {};
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (max(q_begin[mid], 0) / span + mid <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int j = slot - (max(q_begin[lo], 0) / span + lo);
  int r0, r1;
  if (!packed_range(q_begin, lo, a.rows, &r0, &r1, p.status, true) || j < 0) return t;
  if (j >= (r1 - r0 + span - 1) / span) return t;
  const int len = p.seq_lens[lo];
  if (len < 1 || len > p.cap || r1 - r0 > len) {
    report(p.status, kDevBadSeqLen);
    return t;
  }
  t.row0 = r0 + j * span;
  t.ntok = min(span, r1 - t.row0);
  t.seq = lo;
  t.pos0 = len - (r1 - r0) + j * span;
  t.kv1 = t.pos0 + t.ntok;
  t.blocks = (t.kv1 + kBlock - 1) / kBlock;
  return t;
}

// What entry i of a batch in groups is: its group, whether it takes part.
struct Entry {
  int g, g0, g1, first, seq, n, shared;
};

__device__ bool group_entry(const Params& p, const AttendArgs& a, int i, Entry* e) {
  int lo = 0, hi = a.n_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.group_begin[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  e->g = lo;
  e->g0 = a.group_begin[lo];
  e->g1 = a.group_begin[lo + 1];
  const int sb = a.shared_blocks[lo];
  if (e->g1 == e->g0 || i >= e->g1) {
    if (e->g1 < e->g0) report(p.status, kDevBadRange);
    return false;  // entries behind the last group take no part
  }
  if (e->g0 < 0 || e->g0 > i || e->g1 > a.n_members || sb < 0 || sb > p.maxnb) {
    report(p.status, kDevBadRange);
    return false;
  }
  e->seq = a.members[i];
  e->first = a.members[e->g0];
  if (e->seq < 0 || e->seq >= p.B || (sb > 0 && (e->first < 0 || e->first >= p.B))) {
    report(p.status, kDevBadRange);
    return false;
  }
  e->n = p.seq_lens[e->seq];
  const int fn = sb > 0 ? p.seq_lens[e->first] : e->n;  // the prefix is read through the first member
  if (e->n < 0 || e->n > p.cap || fn < 0 || fn > p.cap) {
    report(p.status, kDevBadSeqLen);
    return false;
  }
  const long long shared = static_cast<long long>(sb) * p.bs;
  if (shared > e->n || shared > fn) {
    report(p.status, kDevBadRange);
    return false;
  }
  e->shared = static_cast<int>(shared);
  return true;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ Params p,
                                                            const __grid_constant__ AttendArgs a,
                                                            const __grid_constant__ Plan plan, int slots, int max_ctas) {
  __shared__ long long s_prefix[kPlanSlots + 1];
  __shared__ int s_begin[kPlanSeqs + 1];
  grid_launch_next();
  const int span = 2 * sub_tokens(p.G);
  const int* q_begin = a.q_begin;
  if (q_begin && p.B <= kPlanSeqs) {
    for (int b = threadIdx.x; b <= p.B; b += kPlanThreads) s_begin[b] = q_begin[b];
    q_begin = s_begin;
    __syncthreads();
  }
  long long* prefix = slots <= kPlanSlots ? s_prefix : plan.prefix;
  long long sum = 0;
  for (int base = 0; base < slots; base += kPlanThreads) {
    const int slot = base + threadIdx.x;
    Tile t = {};
    if (slot < slots) {
      if (a.q_begin) {
        t = prompt_tile(p, a, q_begin, slot, span);
      } else if (slot < a.n_members) {  // own tokens of entry `slot`
        Entry e;
        const bool ok = group_entry(p, a, slot, &e);
        plan.row[slot] = ok ? e.seq : -1;
        if (ok && e.n > e.shared) {
          t.row0 = slot;
          t.ntok = 1;
          t.seq = e.seq;
          t.kv0 = e.shared;
          t.kv1 = e.n;
          t.pos0 = kNoMask;
          t.blocks = (t.kv1 - t.kv0 + kBlock - 1) / kBlock;
          t.part0 = (a.n_members + slot) * p.Hq;
        }
      } else {  // shared prefix: the slot of the entry that leads `span` entries of its group
        const int i = slot - a.n_members;
        Entry e;
        // an entry that takes no part itself still leads the others
        int lo = 0, hi = a.n_groups - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (a.group_begin[mid] <= i) lo = mid;
          else hi = mid - 1;
        }
        const int g0 = a.group_begin[lo], g1 = a.group_begin[lo + 1], sb = a.shared_blocks[lo];
        if (g0 >= 0 && g0 <= i && i < g1 && g1 <= a.n_members && sb > 0 && sb <= p.maxnb && (i - g0) % span == 0) {
          const int first = a.members[g0];
          if (first >= 0 && first < p.B && group_entry(p, a, g0, &e)) {
            t.row0 = i;
            t.ntok = min(span, g1 - i);
            t.seq = first;
            t.kv1 = sb * p.bs;
            t.pos0 = kNoMask;
            t.blocks = (t.kv1 + kBlock - 1) / kBlock;
            t.part0 = i * p.Hq;
          }
        }
      }
      plan.tile[slot] = t;
    }
    long long total;
    const long long at = sum + cta_scan<long long>(t.blocks, &total);
    if (slot < slots) plan.prefix[slot] = prefix[slot] = at;
    sum += total;
  }
  if (threadIdx.x == 0) plan.prefix[slots] = sum;
  __syncthreads();
  const long long units = sum * p.Hkv;
  const int ctas = static_cast<int>(min(static_cast<long long>(max_ctas), units));
  if (threadIdx.x == 0) *plan.head = PlanHead{sum, slots, ctas};
  for (int c = threadIdx.x; c < max_ctas; c += kPlanThreads) {
    if (c >= ctas) {
      plan.start[c] = Start{0, 0, 0, slots, 0, 0, {}};
      continue;
    }
    const long long g = first_unit(units, ctas, c);
    const int head = static_cast<int>(g / sum);
    const long long r = g - head * sum;
    int lo = 0, hi = slots - 1;  // the last tile that begins at or before r: not an empty one
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= r) lo = mid;
      else hi = mid - 1;
    }
    const Tile t = plan.tile[lo];
    const int off = static_cast<int>(r - prefix[lo]);
    const int pieces = off > 0 && cta_of(units, ctas, g - off) == c - 1
                           ? cta_of(units, ctas, g - off + t.blocks - 1) - c + 2 : 0;
    plan.start[c] = Start{head, lo, off, slots, first_unit(units, ctas, c + 1) - g, pieces, 0, t};
  }
}

// ------------------------------------------------------------------ walking a CTA's run

struct Piece {
  Tile t;
  int head;
  int b0, b1;   // blocks of the tile
  bool whole;   // this CTA has all of the tile
  bool first;   // ... has its first block

  __device__ __forceinline__ int steps() const {  // of kStep tokens
    return (min(t.kv1 - t.kv0, b1 * kBlock) - b0 * kBlock + kStep - 1) / kStep;
  }
  // Up to 128 rows: both halves take them, half t every other step from t on, and merge at the end.
  __device__ __forceinline__ bool split(int tps) const { return t.ntok <= tps; }
};

struct Walk {
  const Tile* tiles;
  long long left;
  int count, head, tile, off;
  Tile ahead;  // tile `tile`, on its way before it is needed

  __device__ Walk(const Plan& plan, int c) : tiles(plan.tile) {
    const Start s = plan.start[c];
    left = s.left;
    count = s.count;
    head = s.head;
    tile = s.tile;
    off = s.off;
    ahead = s.first;
  }

  __device__ __forceinline__ bool next(Piece* x) {
    while (left > 0) {
      x->t = ahead;
      const int take = static_cast<int>(min(left, static_cast<long long>(x->t.blocks - off)));
      x->head = head;
      x->b0 = off;
      x->b1 = off + take;
      x->first = off == 0;
      x->whole = take == x->t.blocks;
      left -= take;
      off = 0;
      if (++tile == count) {
        tile = 0;
        ++head;
      }
      ahead = tiles[tile];
      if (take > 0) return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ the attention kernel

template <int D>
struct Smem {
  static constexpr int Q_TILE = 128 * D * 2;      // 128 rows of Q
  static constexpr int Q_SLAB = 128 * 128;        // 64 channels of them
  static constexpr int TILE = kStep * D * 2;      // K or V of one step
  static constexpr int SLAB = kStep * 128;
  static constexpr int STAGES = D == 128 ? 9 : 18;
  static constexpr int Q = 0;
  static constexpr int KV = 2 * Q_TILE;
  static constexpr int OUT = KV + STAGES * TILE;  // 32 rows of 64 bytes for each softmax warp
  static constexpr int BARS = OUT + 8 * 2048;
  static constexpr int BYTES = BARS + 768;
};

struct Bars {
  uint64_t full[18], empty[18], clean[18];  // of the stages; clean: rows of V past the last token are zero
  uint64_t s_full[2][2], p_full[2][2];  // [half t][buffer]
  uint64_t turn[4][2];                  // [warp of a half][half t]
  uint64_t xchg[4][2];                  // [warp of a half][half t]
  uint64_t q_full[2], q_free[2], o_step[2], o_full[2], o_free[2], drain[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 768, "barriers fit behind the stages");

// Bounded wait of the kernel's roles, by whole warps; one that gives up makes all give up.
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t phase, volatile int* abort, int* status) {
  bool ok = mbar_try_wait(bar, phase);
  if (__all_sync(0xFFFFFFFFu, ok)) return true;
  const uint64_t t0 = global_ns();
  while (!ok) {
    ok = mbar_try_wait(bar, phase);
    if (ok || *abort) break;
    if (global_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      report(status, kDevWaitTimeout);
    }
  }
  return __all_sync(0xFFFFFFFFu, ok);
}

// The same for a single thread.
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t phase, volatile int* abort, int* status) {
  if (mbar_try_wait(bar, phase)) return true;
  const uint64_t t0 = global_ns();
  while (!mbar_try_wait(bar, phase)) {
    if (*abort) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      report(status, kDevWaitTimeout);
      return false;
    }
  }
  return true;
}

// A position in the ring of stages.
template <int N>
struct Ring {
  int s = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void skip(int n) {
    ph ^= static_cast<uint32_t>((s + n) / N) & 1;
    s = (s + n) % N;
  }
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      ph ^= 1;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p,
                  const __grid_constant__ AttendArgs a, const __grid_constant__ Plan plan) {
  using L = Smem<D>;
  constexpr int NS = L::STAGES, NREG = D / 64;
  constexpr uint32_t S_COL = 0, O_COL = 256, TMEM_COLS = 512;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars& bars = *reinterpret_cast<Bars*>(smem + L::BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G, tps = sub_tokens(G);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], 2);  // both halves have used it
      mbar_init(&bars.clean[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars.s_full[t][i], 1);
        mbar_init(&bars.p_full[t][i], 4);
      }
      mbar_init(&bars.q_full[t], a.q_begin ? 1 : 32);
      mbar_init(&bars.q_free[t], 1);
      mbar_init(&bars.o_step[t], 1);
      mbar_init(&bars.o_full[t], 1);
      mbar_init(&bars.o_free[t], 8);
      mbar_init(&bars.drain[t], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&bars.xchg[i >> 1][i & 1], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&bars.turn[i >> 1][i & 1], 1);
    bars.abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == 8) {
    tmem_alloc(&bars.tmem, TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile int* abort = &bars.abort;
  grid_wait();
  Walk walk(plan, blockIdx.x);
  Piece x;
  bool ok = true;

  if (warp == 10) {
    // ---------------------------------------------------------------- copies: K0 K1 V0 K2 V1 K3 ... (rounds)
    // Each lane works out every 32nd copy, table look-up included, and they issue them in turn: a copy costs its
    // wait and its issue only.
    Ring<NS> ring, mine;  // mine: this lane's last copy
    bool any = false;
    const int bs_log2 = p.bs == 128 ? 7 : 6;
    while (ok && walk.next(&x)) {
      const int begin = x.t.kv0 + x.b0 * kBlock, n = x.steps();
      const bool split = x.split(tps);
      const int rounds = split ? (n + 1) / 2 : n;  // a round: a step for each half, or one for both
      for (int base = 0; ok && base < 2 * n; base += 32) {
        int i = base + lane, sub = 0;
        if (split && n > 1) {
          if ((n & 1) && i > 4 * rounds - 6) ++i;  // the last round is one step: K's has no second
          sub = i & 1;
          i >>= 1;
        }
        const bool v = !(i == 0 || (i & 1 && i < 2 * rounds - 1));  // one round of K ahead of V
        const int round = v ? (i == 2 * rounds - 1 ? rounds - 1 : i / 2 - 1) : (i + 1) / 2;
        const int tok0 = begin + (split ? 2 * round + sub : round) * kStep;
        int row = tok0, slice = x.t.seq * p.Hkv + x.head;
        if (p.table && base + lane < 2 * n) {
          const int blk = tok0 >> bs_log2;
          const int pg = p.table[static_cast<size_t>(x.t.seq) * p.maxnb + blk];
          const bool good = pg >= 0 && pg < p.pages;
          if (!good) report(p.status, kDevBadRange);
          slice = good ? pg * p.Hkv + x.head : p.pages * p.Hkv;  // past the map: zeros
          row = tok0 - (blk << bs_log2);
        }
        const CUtensorMap* map = v ? &vmap : &kmap;
        const int count = min(32, 2 * n - base);
        for (int k = 0; k < count; ++k, ring.next()) {
          if (lane == k) {
            ok = thread_wait(&bars.empty[ring.s], ring.ph ^ 1, abort, p.status);
            if (ok) {
              unsigned char* dst = smem + L::KV + ring.s * L::TILE;
              mbar_expect_tx(&bars.full[ring.s], L::TILE);
              tma_load_4d(dst, map, &bars.full[ring.s], 0, row, 0, slice);
              mine = ring;
              any = true;
            }
          }
          __syncwarp();
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
    }
    // copies still in flight (the last of some lanes) land before the CTA ends; all have, unless a wait ran out
    if (*abort && any) mbar_wait(&bars.full[mine.s], mine.ph, p.status);
    __syncwarp();
  } else if (warp >= 8 && warp < 10) {
    // ---------------------------------------------------------------- products of half t, by one thread
    const int t = warp - 8;
    // a negative scale negates Q, so that the largest product has the largest logit
    const uint32_t QK = mma_desc(128, kStep, false) | (p.scale_log2 < 0.f ? 1u << 13 : 0u);
    constexpr uint32_t PV = mma_desc(128, D, true);
    const uint64_t dQ = tile_desc(smem_addr(smem + L::Q), 16, 1024);
    const uint64_t dK = tile_desc(smem_addr(smem + L::KV), 16, 1024), dV = tile_desc(smem_addr(smem + L::KV), L::SLAB, 1024);
    uint32_t qph = 0, fph = 1, cph = 0;  // phases: Q full, O free; V clean, a bit for each stage
    uint32_t asked = 0, used = 0;         // steps whose S has been asked for, whose P has been used
    Ring<NS> ring;
    // (descriptors differ in their low words, by address / 16: no more than an addition for each product)
    auto qk = [&](int stage, uint32_t buf) {
      const uint64_t q = dQ + t * (L::Q_TILE >> 4), k0 = dK + static_cast<uint32_t>(stage) * (L::TILE >> 4);
      const uint32_t d = tmem + S_COL + t * 128 + buf * 64;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(d, q + ((k / 4) * (L::Q_SLAB >> 4) + (k % 4) * 2), k0 + ((k / 4) * (L::SLAB >> 4) + (k % 4) * 2), QK, k > 0);
    };
    auto pv = [&](int stage, uint32_t buf, bool add) {
      const uint64_t v0 = dV + static_cast<uint32_t>(stage) * (L::TILE >> 4);
      const uint32_t d = tmem + O_COL + t * D, pt = tmem + S_COL + t * 128 + buf * 64;
#pragma unroll
      for (int k = 0; k < kStep / 16; ++k) mma_ts(d, pt + k * 8, v0 + k * 128, PV, add || k > 0);
    };
    if (elect_one()) {
      Ring<NS> other;  // a stage of the other half, still to be let pass
      bool owes = false;
      int last = 0;    // the last stage of the round taken last
      while (ok && walk.next(&x)) {
        const int n = x.steps();
        const bool split = x.split(tps);
        const int rounds = split ? (n + 1) / 2 : n, mine = split ? (n + 1 - t) / 2 : n;
        const bool tail = (x.t.kv1 - x.t.kv0 - x.b0 * kBlock) - (n - 1) * kStep < kStep;
        auto pass = [&](const Ring<NS>& r) {
          ok = ok && thread_wait(&bars.full[r.s], r.ph, abort, p.status);
          if (ok) mbar_arrive(&bars.empty[r.s]);
        };
        // This half's stage of K or V round i, once it has landed.  The other half's stage passes: one ahead of it at
        // once, one behind it before the next is taken.
        auto take = [&](int i) {
          if (owes) pass(other);
          owes = false;
          const bool two = split && 2 * i + 1 < n;
          if (split && t == 1) {
            pass(ring);
            last = ring.s;
            ring.next();
            if (!two) return 0;
          }
          const int stage = last = ring.s;
          ok = ok && thread_wait(&bars.full[ring.s], ring.ph, abort, p.status);
          ring.next();
          if (two && t == 0) {
            other = ring;
            owes = true;
            last = ring.s;
            ring.next();
          }
          return stage;
        };
        ok = thread_wait(&bars.q_full[t], qph, abort, p.status);
        qph ^= 1;
        if (mine == 0) mbar_arrive(&bars.q_free[t]);
        for (int i = 0; ok && i < min(2, rounds); ++i) {  // S of the first two steps
          const int k = take(i);
          if (!ok || i >= mine) break;
          tc_fence_after();
          qk(k, asked & 1);
          tc_commit(&bars.s_full[t][asked & 1]);
          if (i == mine - 1) tc_commit(&bars.q_free[t]);
          tc_commit(&bars.empty[k]);
          ++asked;
        }
        // the previous piece's O has been read
        ok = ok && thread_wait(&bars.o_free[t], fph, abort, p.status);
        fph ^= 1;
        // without a step here the piece could end before that wait, and its phase pass unseen: the softmax threads
        // wait for this
        if (ok && mine == 0) mbar_arrive(&bars.o_full[t]);
        for (int i = 0; ok && i < rounds; ++i) {
          const bool more = i + 2 < mine;
          const uint32_t buf = used & 1;
          const int v = take(i);
          const int at = last;
          const int k2 = i + 2 < rounds ? take(i + 2) : 0;
          if (i == rounds - 1 && tail) {  // `at` is the piece's last stage
            if (ok && (split ? 2 * i + t == n - 1 : true))
              ok = thread_wait(&bars.clean[at], (cph >> at) & 1, abort, p.status);
            cph ^= 1u << at;
          }
          if (!ok || i >= mine) break;
          ok = thread_wait(&bars.p_full[t][buf], (used >> 1) & 1, abort, p.status);
          if (!ok) break;
          tc_fence_after();
          pv(v, buf, i > 0);
          tc_commit(&bars.o_step[t]);
          if (more) {
            qk(k2, buf);  // runs behind the product that reads P there
            tc_commit(&bars.s_full[t][buf]);
            if (i + 3 == mine) tc_commit(&bars.q_free[t]);
            tc_commit(&bars.empty[k2]);
            ++asked;
          } else if (i == mine - 1) {
            tc_commit(&bars.o_full[t]);
          }
          tc_commit(&bars.empty[v]);
          ++used;
        }
      }
      if (owes && ok) {
        ok = thread_wait(&bars.full[other.s], other.ph, abort, p.status);
        if (ok) mbar_arrive(&bars.empty[other.s]);
      }
      if (*abort) {  // products still in flight end before their memory is given back
        tc_commit(&bars.drain[t]);
        mbar_wait(&bars.drain[t], 0, p.status);
      }
    }
    __syncwarp();
  } else if (warp == 11) {
    // ---------------------------------------------------------------- rows of Q; the last rows of V
    uint32_t fph = 3;  // phases, bit t for rows t
    Ring<NS> ring;     // the stage behind the piece's last
    Ring<NS> v;        // the stage of its last V
    int valid = kStep;
    // Rows past the last token may hold anything, and 0 * NaN is not 0.  (Called once the piece's last product
    // with Q is through: the stage's phase is then not ambiguous.)
    auto clean = [&] {
      ok = ok && role_wait(&bars.full[v.s], v.ph, abort, p.status);
      if (!ok) return;
      for (int i = valid * 8 + lane; i < kStep * 8; i += 32)
#pragma unroll
        for (int r = 0; r < NREG; ++r)
          *reinterpret_cast<uint4*>(smem + L::KV + v.s * L::TILE + r * L::SLAB + i * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.clean[v.s]);
    };
    while (ok && walk.next(&x)) {
      const int n = x.steps();
      for (int t = 0; ok && t < 2; ++t) {
        const int tok0 = x.split(tps) ? 0 : t * tps, ntok = min(tps, x.t.ntok - tok0);
        ok = role_wait(&bars.q_free[t], (fph >> t) & 1, abort, p.status);
        fph ^= 1u << t;
        if (ok && t == 0 && valid < kStep) clean();  // of the piece before
        if (!ok) break;
        if (a.q_begin) {  // packed rows: G heads of tps tokens are one box (rows behind the tile's reach no other's result)
          if (lane == 0) {
            mbar_expect_tx(&bars.q_full[t], NREG * 128 * G * tps);
#pragma unroll
            for (int r = 0; r < NREG; ++r)
              tma_load_3d(smem + L::Q + t * L::Q_TILE + r * L::Q_SLAB, &qmap, &bars.q_full[t], r * 64, x.head * G,
                          x.t.row0 + tok0);
          }
          __syncwarp();
          continue;
        }
        // 16-byte chunk c of row r, swizzled as the products read it; rows of no one keep what is there,
        // which reaches no other row's result
        constexpr int C = D / 8, STEP = 32 / C;
        const int c = lane % C;
        const uint16_t* q = a.q + static_cast<size_t>(x.head) * G * D + c * 8;
        const uint32_t dst = smem_addr(smem + L::Q + t * L::Q_TILE + (c >> 3) * L::Q_SLAB);
        int tok = (lane / C) / G, g = (lane / C) % G;
        const int rows = ntok * G;
#pragma unroll 4
        for (int r = lane / C; r < rows; r += STEP) {
          const int row = plan.row[x.t.row0 + tok0 + tok];
          if (row >= 0)
            cp_async_16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                        q + static_cast<size_t>(row) * a.q_stride + static_cast<size_t>(g) * D);
          g += STEP;
          while (g >= G) {
            g -= G;
            ++tok;
          }
        }
        cp_async_wait_all();
        fence_proxy_async();
        mbar_arrive(&bars.q_full[t]);
        __syncwarp();
      }
      ring.skip(2 * n - 1);
      v = ring;
      ring.next();
      valid = (x.t.kv1 - x.t.kv0 - x.b0 * kBlock) - (n - 1) * kStep;
    }
    if (ok && valid < kStep) {
      ok = role_wait(&bars.q_free[0], fph & 1, abort, p.status);
      if (ok) clean();
    }
    __syncwarp();
    if (*abort && a.q_begin && lane == 0)  // a copy in flight lands
      for (int t = 0; t < 2; ++t) mbar_wait(&bars.q_full[t], (fph >> t) & 1, p.status);
  } else {
    // ---------------------------------------------------------------- softmax, rows t
    const int t = warp >> 2, tid = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + S_COL + t * 128 + lanes, tO = tmem + O_COL + t * D + lanes;
    const int tok = tid / G, g = tid - tok * G;
    // scale 0: every logit 0, and a masked one still -infinity
    const float scale = fmaxf(fabsf(p.scale_log2), 1e-30f);
    const float2 sc = make_float2(scale, scale);
    uint32_t step = 0, oph = 0;  // steps of these rows, over all pieces
    uint32_t turn = 0;           // ... with both halves at work
    while (ok && walk.next(&x)) {
      const bool split = x.split(tps);
      const int tok0 = split ? 0 : t * tps, ntok = min(tps, x.t.ntok - tok0);
      const int n = split ? (x.steps() + 1 - t) / 2 : x.steps();  // steps of this half
      const bool mine = tok < ntok;
      const bool work = __any_sync(0xFFFFFFFFu, mine);
      const int e = x.t.row0 + tok0 + (mine ? tok : 0);
      const int row = !mine ? -1 : a.q_begin ? e : plan.row[e];
      // one past the last token this row reads, from this half's next step; rows of no one read all
      int lim = !mine ? kNoMask : (x.t.pos0 == kNoMask ? x.t.kv1 : x.t.pos0 + tok0 + tok + 1) -
                                      (x.t.kv0 + x.b0 * kBlock) - (split ? t * kStep : 0);
      const int stride = split ? 2 * kStep : kStep;
      int least = __reduce_min_sync(0xFFFFFFFFu, lim);  // of the warp's rows
      // The two warps of a scheduler, one of each half, take turns at the exponentials: one loads, looks for its
      // maximum and hands over P while the other has the exponential unit.  Two warps at it at once finish
      // together and then both leave it idle (prompt of 8K, 32/8 heads, d 128: 990 TFLOP/s without turns, 1072 with).
      const bool turns = !split;
      float m = -INFINITY, sum = 0.f;
      for (int j = 0; j < n; ++j, lim -= stride, least -= stride, ++step) {
        const uint32_t buf = step & 1;
        ok = role_wait(&bars.s_full[t][buf], (step >> 1) & 1, abort, p.status);
        if (!ok) break;
        tc_fence_after();
        if (work) {
          const uint32_t tB = tS + buf * 64;
          float s[kStep];
          tmem_ld32(tB, s);
          tmem_ld32(tB + 32, s + 32);
          tmem_wait_ld32(s);
          tmem_wait_ld32(s + 32);
          if (least < kStep) {
#pragma unroll
            for (int c = 0; c < kStep; ++c)
              if (c >= lim) s[c] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < kStep - 4; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], s[c + i], s[c + 4 + i]);
          const float m1 = fmaxf(m, max3(max3(mx[0], mx[1], s[kStep - 4]), max3(mx[2], mx[3], s[kStep - 3]),
                                         fmaxf(s[kStep - 2], s[kStep - 1])) * scale);
          if (j == 0) {
            m = m1;
          } else if (__any_sync(0xFFFFFFFFu, mine && (m1 - m > kGrow || (m == -INFINITY && m1 > m)))) {
            // O holds the steps before this one once the last product is through.  (S of this
            // step came behind the product two steps back, so the phase is not ambiguous.)
            ok = role_wait(&bars.o_step[t], (step - 1) & 1, abort, p.status);
            if (!ok) break;
            tc_fence_after();
            const float f = m1 == -INFINITY ? 1.f : exp2_fast(m - m1);
            m = m1;
            sum *= f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_ld32(tO + c, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f;
              tmem_st32(tO + c, o);
            }
          }
          if (turns) ok = role_wait(&bars.turn[warp & 3][t], (turn & 1) ^ (t ^ 1), abort, p.status);
          if (!ok) break;
          const float base = m == -INFINITY ? 0.f : m;
          const float2 off = make_float2(-base, -base);
          float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < kStep / 32; ++h) {
            uint32_t w[16];
            float2 y[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) y[c] = fma2(make_float2(s[h * 32 + 2 * c], s[h * 32 + 2 * c + 1]), sc, off);
#pragma unroll
            for (int c = 0; c < 16; ++c) y[c] = make_float2(exp2_fast(y[c].x), exp2_fast(y[c].y));
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              part[c & 1] = add2(part[c & 1], y[c]);
              w[c] = pack_bf16(y[c].x, y[c].y);
            }
            tmem_st16(tB + h * 16, w);
          }
          if (turns && lane == 0) mbar_arrive(&bars.turn[warp & 3][t ^ 1]);
          sum += (part[0].x + part[1].x) + (part[0].y + part[1].y);
          tmem_wait_st();
        } else if (turns) {
          ok = role_wait(&bars.turn[warp & 3][t], (turn & 1) ^ (t ^ 1), abort, p.status);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&bars.turn[warp & 3][t ^ 1]);
        }
        turn += turns;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[t][buf]);
      }
      ok = ok && role_wait(&bars.o_full[t], oph, abort, p.status);
      oph ^= 1;
      if (!ok) break;
      tc_fence_after();
      unsigned char* box = smem + L::OUT + warp * 2048;
      float f = 1.f, fo = 0.f;  // factors of this half's and the other half's O, in a split piece
      if (split) {              // (by warps without rows too: none gets a piece ahead of its partner)
        uint64_t* here = &bars.xchg[warp & 3][t];
        uint64_t* there = &bars.xchg[warp & 3][t ^ 1];
        reinterpret_cast<float2*>(box)[lane] = make_float2(m, sum);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(there);
        ok = role_wait(here, 0, abort, p.status);
        if (!ok) break;
        tc_fence_after();  // the other half's O is complete too
        const float2 o = reinterpret_cast<const float2*>(smem + L::OUT + (warp ^ 4) * 2048)[lane];
        __syncwarp();
        if (lane == 0) mbar_arrive(there);
        const float both = fmaxf(m, o.x);
        f = sum == 0.f ? 0.f : exp2_fast(m - both);
        fo = o.y == 0.f ? 0.f : exp2_fast(o.x - both);
        m = both;
        sum = sum * f + o.y * fo;
        ok = role_wait(here, 1, abort, p.status);  // the other half has read the box
        if (!ok) break;
      }
      if (work) {
        const int hq = x.head * G + g;
        const bool direct = a.q_begin && x.whole;
        const float inv = 1.f / sum;  // (a row of a whole tile has tokens: 0 / 0 where every score is -infinity)
        const size_t at = static_cast<size_t>(row < 0 ? 0 : row) * p.Hq + hq;
        // partial rows: of the CTA (a tile's later pieces; of a prompt also its first), or of the batch
        const int prow0 = (split ? 0 : t * 128) + tid;
        const size_t prow = !x.first ? (2ull * blockIdx.x) * 256 + prow0
                            : a.q_begin ? (2ull * blockIdx.x + 1) * 256 + prow0
                                        : 2ull * kMaxAttendCtas * 256 + x.t.part0 +
                                              static_cast<size_t>(tok0 + tok) * p.Hq + hq;
        float* part = plan.part + prow * (D + 4);
        if (row >= 0 && !(split && t == 1)) {
          if (!direct) {
            part[0] = m;
            part[1] = sum;
          } else if (a.lse) {
            a.lse[at] = (m + log2f(sum)) * 0.6931471805599453f;
          }
        }
        // Each thread has one row; 64 bytes of the warp's rows at a time go through shared memory, so
        // that four threads store 64 consecutive bytes of a row; few rows go straight out.  (No row straight out, up to
        // 16, all: 64 sequences on four prefixes of 128K 471, 457, 451 us; 16 on one of 16K, one head a group, 51, 47,
        // 47; 16 ragged prompts 88, 88, 96; one of 2048 rows 82, 82, 88; 256 of 64 tokens each on four prefixes of 1K
        // 104, 104, 108.)
        char* own = row < 0 ? nullptr : direct ? reinterpret_cast<char*>(a.out + at * D) : reinterpret_cast<char*>(part + 4);
        char* to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[i] = reinterpret_cast<char*>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(own), 8 * i + lane / 4));
        const bool few = ntok * G <= 16;
        auto store64 = [&](const uint4 (&w)[4], int offset) {
          if (few) {
            if (own)
#pragma unroll
              for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(own + offset + i * 16) = w[i];
            return;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(box + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = w[i];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + lane / 4;
            const uint4 v = *reinterpret_cast<const uint4*>(box + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
            if (to[i]) *reinterpret_cast<uint4*>(to[i] + offset + (lane & 3) * 16) = v;
          }
        };
        // (of a split piece half the columns each)
#pragma unroll 1
        for (int c = split ? t * (D / 2) : 0; c < (split ? (t + 1) * (D / 2) : D); c += 32) {
          float o[32];
          tmem_ld32(tO + c, o);
          tmem_wait_ld32(o);
          if (split) {
            float q[32];
            tmem_ld32(tmem + O_COL + (t ^ 1) * D + lanes + c, q);
            tmem_wait_ld32(q);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = (f != 0.f ? o[i] * f : 0.f) + (fo != 0.f ? q[i] * fo : 0.f);
          }
          uint4 w[4];
          if (direct) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = make_uint4(pack_bf16(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                pack_bf16(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                pack_bf16(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
            store64(w, c * 2);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = make_uint4(__float_as_uint(o[16 * h + 4 * i]), __float_as_uint(o[16 * h + 4 * i + 1]),
                                  __float_as_uint(o[16 * h + 4 * i + 2]), __float_as_uint(o[16 * h + 4 * i + 3]));
              store64(w, c * 4 + h * 64);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {  // O has been read: both halves', of a split piece, else this half's (both of its arrivals)
        mbar_arrive(&bars.o_free[t]);
        mbar_arrive(&bars.o_free[split ? t ^ 1 : t]);
      }
    }
  }
  __syncthreads();
  grid_launch_next();
  if (warp == 8) {
    tc_fence_after();
    tmem_free(tmem, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ merging partials

constexpr int kMergeWarps = 4;

// Merge the n partial rows that row_of(i) names and write the result.  Few rows: one warp
// (rows of different warps are different results).  With a CTA to every result: 16 ragged prompts 113 us, 88 so; a prompt
// of 2048 rows 111 and 82; 64 sequences on four prefixes of 128K 471 and 457; where most tiles have many pieces (4 prompts of
// 32 rows behind 16K) 80 and 82.
template <int D, int kFewRows, typename RowOf>
__device__ void merge_few(const Plan& plan, const AttendArgs& a, int n, size_t at, RowOf row_of) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  float rm[kFewRows], rs[kFewRows], ro[kFewRows][C];
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    rm[i] = -INFINITY;
    rs[i] = 0.f;
    if (i < n) {
      const float* r = plan.part + row_of(i) * (D + 4);
      rm[i] = r[0];
      rs[i] = r[1];
#pragma unroll
      for (int c = 0; c < C; ++c) ro[i][c] = r[4 + lane * C + c];
    }
  }
  float m = rm[0], sum = 0.f, acc[C];
#pragma unroll
  for (int i = 1; i < kFewRows; ++i) m = fmaxf(m, rm[i]);
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll
  for (int i = 0; i < kFewRows; ++i) {
    if (rs[i] == 0.f) continue;  // nothing there: the rest of the row may hold anything
    const float f = exp2f(rm[i] - m);
    sum += rs[i] * f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] += ro[i][c] * f;
  }
  const float inv = n == 0 ? 0.f : 1.f / sum;  // no piece: a sequence without tokens
#pragma unroll
  for (int c = 0; c < C; c += 2)
    reinterpret_cast<uint32_t*>(a.out + at * D + lane * C)[c / 2] = pack_bf16(acc[c] * inv, acc[c + 1] * inv);
  if (a.lse && lane == 0) a.lse[at] = (m + log2f(sum)) * 0.6931471805599453f;
}

// Many rows: one CTA, its warps taking every kMergeWarps-th, with the loads of four rows under way at a time.
template <int D, typename RowOf>
__device__ void merge_many(const Plan& plan, const AttendArgs& a, int n, size_t at, RowOf row_of) {
  constexpr int C = D / 32;
  __shared__ float s_m[kMergeWarps], s_sum[kMergeWarps], s_acc[kMergeWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = -INFINITY, sum = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  for (int i0 = warp; i0 < n; i0 += 4 * kMergeWarps) {
    float rm[4], rs[4], ro[4][C];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kMergeWarps;
      rm[u] = -INFINITY;
      rs[u] = 0.f;
      if (i < n) {
        const float* r = plan.part + row_of(i) * (D + 4);
        rm[u] = r[0];
        rs[u] = r[1];
#pragma unroll
        for (int c = 0; c < C; ++c) ro[u][c] = r[4 + lane * C + c];
      }
    }
    const float m1 = fmaxf(m, fmaxf(fmaxf(rm[0], rm[1]), fmaxf(rm[2], rm[3])));
    const float f = m == m1 ? 1.f : exp2f(m - m1);  // (the same infinity: nothing to rescale)
    m = m1;
    sum *= f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= f;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (rs[u] == 0.f) continue;  // nothing there: the rest of the row may hold anything
      const float g = exp2f(rm[u] - m);
      sum += rs[u] * g;
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += ro[u][c] * g;
    }
  }
  __syncthreads();  // the row before has been read
  if (lane == 0) {
    s_m[warp] = m;
    s_sum[warp] = sum;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) s_acc[warp][lane * C + c] = acc[c];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  m = s_m[0];
  for (int w = 1; w < kMergeWarps; ++w) m = fmaxf(m, s_m[w]);
  float x = 0.f, y = 0.f;
  sum = 0.f;
  for (int w = 0; w < kMergeWarps; ++w) {
    const float f = s_sum[w] == 0.f ? 0.f : exp2f(s_m[w] - m);
    sum += s_sum[w] * f;
    x += s_acc[w][2 * threadIdx.x] * f;
    y += s_acc[w][2 * threadIdx.x + 1] * f;
  }
  const float inv = 1.f / sum;  // (there is a piece, so there are tokens)
  reinterpret_cast<uint32_t*>(a.out + at * D)[threadIdx.x] = pack_bf16(x * inv, y * inv);
  if (a.lse && threadIdx.x == 0) a.lse[at] = (m + log2f(sum)) * 0.6931471805599453f;
}

// Packed prompts: CTA column c merges the tile that was cut first at the start of CTA c's run.
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) combine_tiles_kernel(const __grid_constant__ Params p,
                                                            const __grid_constant__ AttendArgs a,
                                                            const __grid_constant__ Plan plan) {
  const int c = blockIdx.x + 1;
  grid_wait();
  const Start s = plan.start[c];
  const int n = s.pieces, tps = sub_tokens(p.G);
  if (n == 0) return;
  const Tile& t = s.first;
  constexpr int kFewRows = 4;
  const bool few = n <= kFewRows;
  const int warp = few ? threadIdx.x >> 5 : 0, warps = few ? kMergeWarps : 1;
  for (int r = blockIdx.y * warps + warp; r < t.ntok * p.G; r += gridDim.y * warps) {
    const int tok = r / p.G, g = r % p.G;
    const int prow = tok / tps * 128 + (tok % tps) * p.G + g;
    const size_t at = static_cast<size_t>(t.row0 + tok) * p.Hq + s.head * p.G + g;
    auto row_of = [&](int i) { return (i == 0 ? 2ull * (c - 1) + 1 : 2ull * (c + i - 1)) * 256 + prow; };
    if (few) merge_few<D, kFewRows>(plan, a, n, at, row_of);
    else merge_many<D>(plan, a, n, at, row_of);
  }
}

// A batch in groups: each query head of an entry is merged from its prefix and its own tokens, by a CTA, or by
// a warp where there are few pieces (the CTAs left over end).
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) combine_entries_kernel(const __grid_constant__ Params p,
                                                                           const __grid_constant__ AttendArgs a,
                                                                           const __grid_constant__ Plan plan) {
  const int i = blockIdx.x;
  grid_wait();
  const int row = plan.row[i];
  if (row < 0) return;
  const PlanHead h = *plan.head;
  const long long units = h.per_head * p.Hkv;
  const int tps = sub_tokens(p.G);
  // the entry's prefix tile is the slot of the entry that leads it
  int lo = 0, hi = a.n_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.group_begin[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  const int lead = i - (i - a.group_begin[lo]) % (2 * tps);
  const int slot[2] = {a.n_members + lead, i};
  const Tile tile[2] = {plan.tile[slot[0]], plan.tile[slot[1]]};
  auto merge = [&](int hq, auto&& how) {
    const int head = hq / p.G, g = hq % p.G;
    int c0[2] = {0, 0}, n[2] = {0, 0};
    size_t first[2], later[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Tile& t = tile[k];
      if (t.blocks == 0) continue;
      const long long z0 = head * h.per_head + plan.prefix[slot[k]];
      c0[k] = cta_of(units, h.ctas, z0);
      n[k] = cta_of(units, h.ctas, z0 + t.blocks - 1) - c0[k] + 1;
      const int tok = i - t.row0;
      first[k] = 2ull * kMaxAttendCtas * 256 + t.part0 + static_cast<size_t>(tok) * p.Hq + hq;
      later[k] = tok / tps * 128 + (tok % tps) * p.G + g;
    }
    how(n[0] + n[1], static_cast<size_t>(row) * p.Hq + hq, [&](int j) {
      const int k = j < n[0] ? 0 : 1, piece = k ? j - n[0] : j;
      return piece == 0 ? first[k] : 2ull * (c0[k] + piece) * 256 + later[k];
    });
  };
  // no head has more pieces than this
  const long long run = units > 0 ? max(units / h.ctas, 1ll) : 1;
  long long most = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) most += tile[k].blocks ? (tile[k].blocks - 1) / run + 2 : 0;
  constexpr int kFewRows = 8;
  const bool few = most <= kFewRows;
  if (few) {
    const int hq = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
    if (hq < p.Hq) merge(hq, [&](int n, size_t at, auto&& row_of) { merge_few<D, kFewRows>(plan, a, n, at, row_of); });
  } else {
    merge(blockIdx.y, [&](int n, size_t at, auto&& row_of) { merge_many<D>(plan, a, n, at, row_of); });
  }
}

// ------------------------------------------------------------------ launches

Plan plan_of(const Params& p, const AttendArgs& a) {
  unsigned char* w = static_cast<unsigned char*>(a.work);
  Plan plan;
  const size_t tiles = attend_tiles(p.B, a.max_rows, p.G);
  auto take = [&](size_t bytes) {
    unsigned char* at = w;
    w += (bytes + 255) & ~static_cast<size_t>(255);
    return at;
  };
  plan.head = reinterpret_cast<PlanHead*>(take(sizeof(PlanHead)));
  plan.start = reinterpret_cast<Start*>(take(sizeof(Start) * kMaxAttendCtas));
  plan.prefix = reinterpret_cast<long long*>(take(8 * (tiles + 1)));
  plan.tile = reinterpret_cast<Tile*>(take(sizeof(Tile) * tiles));
  plan.row = reinterpret_cast<int*>(take(4 * static_cast<size_t>(p.B)));
  plan.part = reinterpret_cast<float*>(w);
  return plan;
}

template <int D>
cudaError_t launch_attend_t(const Params& p, const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, int sms, cudaStream_t s) {
  const Plan plan = plan_of(p, a);
  const int span = 2 * sub_tokens(p.G);
  const int slots = a.q_begin ? a.rows / span + p.B : 2 * a.n_members;
  const int ctas = sms < kMaxAttendCtas ? sms : kMaxAttendCtas;
  cudaError_t e = allow_max_smem(reinterpret_cast<const void*>(attend_kernel<D>));
  if (e == cudaSuccess) e = launch_kernel(plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, 0, p, a, plan, slots, ctas);
  if (e == cudaSuccess)
    e = launch_kernel_early(attend_kernel<D>, dim3(ctas), dim3(kAttendThreads), Smem<D>::BYTES + 1024, s, qmap, kmap, vmap,
                            p, a, plan);
  if (e != cudaSuccess) return e;
  if (!a.q_begin)
    return launch_kernel_early(combine_entries_kernel<D>, dim3(a.n_members, p.Hq), dim3(32 * kMergeWarps), 0, s, p, a, plan);
  if (ctas == 1) return e;
  return launch_kernel_early(combine_tiles_kernel<D>, dim3(ctas - 1, 32), dim3(32 * kMergeWarps), 0, s, p, a, plan);
}

}  // namespace

size_t attend_tiles(int B, int max_rows, int G) {
  const size_t packed = static_cast<size_t>(max_rows / (2 * sub_tokens(G))) + B, grouped = 2 * static_cast<size_t>(B);
  return packed > grouped ? packed : grouped;
}

size_t attend_work_bytes(int B, int Hq, int G, int d, int max_rows) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t tiles = attend_tiles(B, max_rows, G);
  return up(sizeof(PlanHead)) + up(sizeof(Start) * kMaxAttendCtas) + up(8 * (tiles + 1)) + up(sizeof(Tile) * tiles) +
         up(4 * static_cast<size_t>(B)) +
         up((2ull * kMaxAttendCtas * 256 + 2ull * B * Hq) * (d + 4) * sizeof(float));
}

cudaError_t launch_attend(const Params& p, const AttendArgs& a, const CUtensorMap& qmap, const CUtensorMap& kmap,
                          const CUtensorMap& vmap, int sms, cudaStream_t s) {
  return p.d == 128 ? launch_attend_t<128>(p, a, qmap, kmap, vmap, sms, s)
                    : launch_attend_t<64>(p, a, qmap, kmap, vmap, sms, s);
}

}  // namespace prr
