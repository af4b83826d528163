// The backward pass over packed sequences: the gradient kernel (fa_backward.cuh) over
// Q, dO [total, Hq, d] and K, V [total, Hkv, d], and its preprocess kernel.
//
// Blocks are 128-row tiles of the sequences, from the plan's lists. A key block of a
// key/value head runs over the queries of all Hq / Hkv query heads that read it, so
// that dK and dV are summed on chip, in a fixed order, and written once; unless the batch
// has so few key blocks that one would take longer than an SM's share of all the work.
// Then its queries are split into parts, whose fp32 sums a last kernel joins, in order
// (one sequence of 4000 rows, 4/1 heads, d = 128: 82 us, 209 unsplit; 2000 rows, 8/1: 54
// and 220). The statistics -D and -L * log2(e) lie in a workspace in which every sequence
// starts on a multiple of 128 rows: TMA copies of fp32 rows have to start on 16-byte
// boundaries, which a sequence's first row in the packed tensors need not do.
#include "fa_backward.cuh"
#include "fa_launch.h"
#include "fa_packed.cuh"

namespace fa {

__device__ unsigned int g_packed_bwd_status;

namespace {

struct PackedBwdParams {
  const uint8_t* plan;
  long long off_kv, off_q;  // the lists' places in the plan
  __nv_bfloat16 *dQ, *dK, *dV;
  long long lddq, lddk, lddv;
  const float *nD, *nL2;
  const BwdDealHead* deal;
  const BwdItem* items;
  const uint8_t* ranks;
  float* parts;
  long long ws_rows;
  int total, nseq, Hq, Hkv, per_kv, causal, kgroup, qgroup, fill, trigger;
};

// SPLIT: key blocks may have been split and the items dealt by ranks (see deal_items). It
// is a kernel of its own: the look-ups cost the other batches 2 %.
template <bool SPLIT>
struct PackedBwd {
  using Params = PackedBwdParams;
  struct View {
    const Params& p;
    int tiles, covered;
    int4 deal, mine;  // BwdDealHead
  };
  using KvItem = BwdItem;
  struct QItem {
    PlanTile s;
    int h;
  };
  static constexpr bool kEarly = true;
  static constexpr bool kHeads = true, kListed = true, kForeignTail = true;
  FA_DEV static unsigned int* status() { return &g_packed_bwd_status; }
  FA_DEV static bool trigger(const Params& p) { return p.trigger; }
  FA_DEV static View view(const Params& p) {
    const PlanHead* head = reinterpret_cast<const PlanHead*>(p.plan);
    int4 mine = make_int4(0, 0, 0, 0), deal = mine;
    if constexpr (SPLIT) {
      mine = p.deal->cta[blockIdx.x];
      deal = *reinterpret_cast<const int4*>(p.deal);
    }
    const bool ok = plan_matches(head, p.total, p.nseq, status());
    return {p, ok ? head->tiles128 : 0, ok ? head->covered : p.total, deal, mine};
  }
  // Without split key blocks each list is dealt in snake order, the query blocks in reverse
  // CTA order; with them, by the ranks (see deal_items).
  FA_DEV static bool ranked(const View& g) { return SPLIT && g.deal.y > 0; }
  FA_DEV static int causal(const View& g) { return g.p.causal; }
  FA_DEV static int kv_count(const View& g, int c, int P) {
    return ranked(g) ? g.mine.x : snake_count(g.tiles * g.p.Hkv, c, P);
  }
  FA_DEV static int q_count(const View& g, int c, int P) {
    return ranked(g) ? g.mine.y : snake_count(g.tiles * g.p.Hq, P - 1 - c, P);
  }

  FA_DEV static int kv_rank(const View& g, int t, int c, int P) {
    if (!ranked(g)) return 0;
    const int row = t >> (g.deal.w & 255);
    return row == 0 ? c : g.p.ranks[(size_t)row * P + c];
  }
  FA_DEV static int q_rank(const View& g, int t, int c, int P) {
    if (!ranked(g)) return 0;
    const int row = t >> (g.deal.w >> 8);
    return row == 0 ? g.mine.z : g.p.ranks[(size_t)(g.mine.w + row) * P + c];
  }
  FA_DEV static KvItem kv_item(const View& g, int t, int rank, int c, int P) {
    const int i = ranked(g) ? t * P + rank : snake_item(t, c, P);
    if (SPLIT && i < g.deal.x) {
      const int4* e = reinterpret_cast<const int4*>(g.p.items + i);
      const int4 s = e[0], r = e[1];
      return {s, r.x, r.y, r.z, r.w};
    }
    int tile, hk;
    const int from = SPLIT ? g.deal.y : 0;
    grouped_tile(i - (SPLIT ? g.deal.x : 0), g.p.Hkv, g.tiles - from, g.p.kgroup, tile, hk);
    KvItem it;
    it.s = reinterpret_cast<const PlanTile*>(g.p.plan + g.p.off_kv)[from + tile];
    it.head = hk;
    it.first = it.halves = 0;
    it.slot = -1;
    return it;
  }
  FA_DEV static int first_key(const KvItem& it) { return it.s.z * 128; }
  FA_DEV static int rows(const View&, const KvItem& it) { return it.s.y; }
  FA_DEV static int keys(const View&, const KvItem& it) { return it.s.y; }
  FA_DEV static int kv_halves(const View& g, const KvItem& it, int& q_first) {
    q_first = g.p.causal ? it.s.z * 128 : 0;
    return (it.s.y - q_first + 63) / 64;
  }
  FA_DEV static int kv_part(const View& g, const KvItem& it, int per, int& first) {
    first = SPLIT ? it.first : 0;
    return SPLIT && it.halves > 0 ? it.halves : per * g.p.per_kv;
  }
  FA_DEV static void load_keys(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                               const View&, const KvItem& it) {
    tma_load_3d(dst, map, f, col, it.head, it.s.x + it.s.z * 128);
  }
  FA_DEV static void load_queries(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                  const View& g, const KvItem& it, int hd, int q) {
    tma_load_3d(dst, map, f, col, it.head * g.p.per_kv + hd, it.s.x + q);
  }
  FA_DEV static void load_stats(void* dst, const CUtensorMap* map, uint64_t* f, const View& g,
                                const KvItem& it, int hd, int q) {
    tma_load_2d(dst, map, f, it.s.w + q, it.head * g.p.per_kv + hd);
  }
  template <int D>
  FA_DEV static void store_keys(const View& g, const KvItem& it, int w, int warp, uint32_t col,
                                float mul, uint8_t* stage, const CUtensorMap* map, int d) {
    const int key = it.s.z * 128 + warp * 32;
    if (SPLIT && it.slot >= 0) {
      part_store<D>(col, g.p.parts + ((size_t)(2 * it.slot + w) * 4 + warp) * 32 * D, d);
      return;
    }
    packed_rows_store<D>(col, mul, stage, map, it.head, it.s.x + key, it.s.y - key, 0, d,
                         w == 0 ? g.p.dV : g.p.dK, w == 0 ? g.p.lddv : g.p.lddk);
  }
  // Sums of a part: D columns of a warp's 32 rows, four columns of all rows after another
  // (full 128-byte lines; see packed_join_kernel).
  template <int D>
  FA_DEV static void part_store(uint32_t col, float* out, int d) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      if (c >= d) break;  // warp-uniform
      uint32_t o[32];
      tmem_ld32(col + c, o);
      tmem_ld_wait();
      reg_fence32(o);
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<uint4*>(out + ((c + e) * 8 + lane) * 4) =
            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
  }
  template <int D>
  FA_DEV static void zero_key(const View&, const KvItem&, int, int, int) {}  // every key is seen

  FA_DEV static QItem q_item(const View& g, int t, int rank, int c, int P) {
    int tile, h;
    const int i = ranked(g) ? t * P + rank : snake_item(t, P - 1 - c, P);
    grouped_tile(i, g.p.Hq, g.tiles, g.p.qgroup, tile, h);
    return {reinterpret_cast<const PlanTile*>(g.p.plan + g.p.off_q)[tile], h};
  }
  FA_DEV static int first_query(const QItem& it) { return it.s.z * 128; }
  FA_DEV static int keys(const View&, const QItem& it) { return it.s.y; }
  FA_DEV static int key_blocks(const View& g, const QItem& it) {
    return g.p.causal ? it.s.z + 1 : (it.s.y + 127) / 128;
  }
  FA_DEV static void load_block_queries(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                        const View&, const QItem& it, int row) {
    tma_load_3d(dst, map, f, col, it.h, it.s.x + it.s.z * 128 + row);
  }
  FA_DEV static void load_block_keys(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                                     const View& g, const QItem& it, int key) {
    tma_load_3d(dst, map, f, col, it.h / g.p.per_kv, it.s.x + key);
  }
  FA_DEV static void query_stats(const View& g, const QItem& it, int r, float& nl2, float& nd) {
    const size_t row = (size_t)it.h * g.p.ws_rows + it.s.w + it.s.z * 128 + r;
    nl2 = g.p.nL2[row];
    nd = g.p.nD[row];
  }
  template <int NCOL>
  FA_DEV static void store_queries(const View& g, const QItem& it, int warp, uint32_t tcol,
                                   float mul, uint8_t* stage, const CUtensorMap* map, int col0,
                                   int d) {
    const int q = it.s.z * 128 + warp * 32;
    packed_rows_store<NCOL>(tcol, mul, stage, map, it.h, it.s.x + q, it.s.y - q, col0, d, g.p.dQ,
                            g.p.lddq);
  }
  // Rows that no sequence covers, where the caller asked for zeros.
  FA_DEV static void finish(const View& g, int d) {
    const Params& p = g.p;
    const long long t = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long nt = (long long)gridDim.x * blockDim.x;
    if (p.fill & 1) zero_rows(p.dQ, g.covered, p.total, p.Hq * d, p.lddq, t, nt);
    if (p.fill & 2) zero_rows(p.dK, g.covered, p.total, p.Hkv * d, p.lddk, t, nt);
    if (p.fill & 4) zero_rows(p.dV, g.covered, p.total, p.Hkv * d, p.lddv, t, nt);
  }
};

// Splitting key blocks, and the deal of the gradient kernel's items to its CTAs where some
// are split, by one block of the preprocess kernel: first the dK/dV pass, then the dQ pass,
// each in launch order (the heaviest first inside a group of heads), in rounds of one item
// per CTA. The CTA with the least work so far gets a round's first item (its rank is 0); in
// long lists several rounds share their ranks, so that at most 16 times are sorted.
// Larger batches are not dealt so: for 16384 rows in 12 sequences, 32/8 heads, d = 128, the
// busiest CTA came from 9 % above the mean to 2 %, but the mean rose by 2 %, and the deal's
// time was not hidden everywhere (8192 rows in 23, 16/16, d = 64: 168 us, 152 in snake order).
struct DealArgs {
  const uint8_t* plan;
  long long off_kv, off_q;  // the lists' places in the plan
  BwdDealHead* head;
  BwdJoin* joins;
  BwdItem* items;
  uint8_t* ranks;
  int P, Hq, Hkv, causal, kgroup, qgroup, slots;
  int half_cost, kv_cost, block_cost, q_cost;  // time of an item, in about 200 cycles
};

// x / d for 0 <= x < 2^31.
struct Divisor {
  unsigned d, m;
  __device__ explicit Divisor(int n) : d((unsigned)n), m(0xffffffffu / (unsigned)n) {}
  __device__ unsigned operator()(unsigned x) const {
    const unsigned q = __umulhi(x, m);  // the quotient or one less
    return q + (x - q * d >= d ? 1 : 0);
  }
};

__device__ __noinline__ void deal_items(const DealArgs& a, int tiles) {
  constexpr int T = 256;
  constexpr int CACHED = 1024;  // tiles whose work is held in shared memory
  __shared__ int kv_work[CACHED], q_work[CACHED], part_work[kMaxParts];
  __shared__ unsigned bins[T], scan[T / 32], lows[T / 32], highs[T / 32];
  __shared__ long long wide[T / 32];
  __shared__ int split_tiles;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_kv = a.Hq / a.Hkv;
  const PlanTile* kv = reinterpret_cast<const PlanTile*>(a.plan + a.off_kv);
  const PlanTile* qs = reinterpret_cast<const PlanTile*>(a.plan + a.off_q);
  auto halves = [&](const PlanTile& s) { return (s.y - (a.causal ? s.z * 128 : 0) + 63) / 64; };
  auto blocks = [&](const PlanTile& s) { return a.causal ? s.z + 1 : (s.y + 127) / 128; };

  // Work of every tile, and of the batch.
  bins[tid] = 0;
  if (tid == 0) split_tiles = 0;
  long long sum = 0;
  for (int e0 = tid; e0 < tiles; e0 += 4 * T) {
    PlanTile k[4], q[4];  // loads of four rounds before the first store
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = min(e0 + u * T, tiles - 1);
      k[u] = kv[e];
      q[u] = qs[e];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = e0 + u * T;
      if (e >= tiles) break;
      const int h = halves(k[u]);
      sum += h;
      if (e < CACHED) {
        kv_work[e] = h;
        q_work[e] = blocks(q[u]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) wide[warp] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int i = 0; i < T / 32; ++i) sum += wide[i];
  const long long share = (sum * a.Hq * 6 + 5 * kPartShare - 1) / (5 * kPartShare);
  const int hc = (int)max((long long)kMinPart, min(share, 0x7fffffffLL));

  // The tiles to split are the list's first: it is in order of their 128-query blocks, so up
  // to one half. (The ones before the last of them that have a half less stay whole, as one
  // part: what is split does not depend on the order of equals, which is not fixed. They
  // have more than 5/6 hc halves.)
  int last = 0;
  for (int e = tid; e < tiles; e += T)
    if ((long long)(e < CACHED ? kv_work[e] : halves(kv[e])) * per_kv * 3 > hc * 5LL)
      last = e + 1;
  if (last > 0) atomicMax(&split_tiles, last);
  __syncthreads();
  int n_split = split_tiles;
  if ((long long)n_split * a.Hkv > T) n_split = 0;  // cannot be: see kMaxParts
  int n_parts = 0, joins = 0;
  if (n_split > 0) {
    BwdItem it{};
    int parts = 0;
    if (tid < n_split * a.Hkv) {
      it.head = tid % a.Hkv;
      it.s = kv[tid / a.Hkv];
      it.halves = halves(it.s) * per_kv;
      parts = it.halves * 3LL > hc * 5LL ? (it.halves - 1) / hc + 1 : 1;
    }
    // Items in bits 0..9, slots in 10..19, joins in 20..29.
    const unsigned add = parts > 1 ? (unsigned)parts * 1025u + (1u << 20) : (unsigned)parts;
    unsigned inc = add;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    unsigned all = 0;
#pragma unroll
    for (int i = 0; i < T / 32; ++i) {
      if (i < warp) inc += scan[i];
      all += scan[i];
    }
    inc -= add;
    n_parts = (int)(all & 1023u);
    joins = (int)(all >> 20);
    if (n_parts > a.slots) n_split = n_parts = joins = 0;  // cannot be, either
    if (n_parts > 0 && parts > 0) {
      const int at = (int)(inc & 1023u), slot = (int)((inc >> 10) & 1023u), nu = it.halves;
      if (parts > 1) a.joins[inc >> 20] = {it.s, it.head, slot, parts, 0};
      for (int k = 0; k < parts; ++k) {
        it.first = (int)((long long)nu * k / parts);
        it.halves = (int)((long long)nu * (k + 1) / parts) - it.first;
        it.slot = parts > 1 ? slot + k : -1;
        a.items[at + k] = it;
        part_work[at + k] = it.halves;
      }
    }
    __syncthreads();
  }

  if (n_split == 0) {
    if (tid == 0) *reinterpret_cast<int4*>(a.head) = make_int4(0, 0, 0, 0);
    return;
  }

  unsigned load = 0;  // of CTA tid
  int4 mine = make_int4(0, 0, tid, 0);
  int row_of_ranks = 0, shifts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    const int heads = pass == 0 ? a.Hkv : a.Hq, from = pass == 0 ? n_split : 0;
    const int group = pass == 0 ? a.kgroup : a.qgroup, head_items = pass == 0 ? n_parts : 0;
    const int n = head_items + (tiles - from) * heads, rounds = (n + a.P - 1) / a.P;
    int shift = 0;
    while (rounds >> shift > 8) ++shift;
    int taken = 0;
    if (pass == 1) mine.w = row_of_ranks;
    const int groups = (heads + group - 1) / group;
    const Divisor per_group(max(1, group * (tiles - from))), per_tile(group),
        per_last(heads - (groups - 1) * group);
    for (int round = 0; round < rounds; round += 1 << shift, ++row_of_ranks) {
      int rank = tid;
      if (row_of_ranks > 0) {
        // Rank of CTA tid by its work so far: a counting sort over 256 classes of it.
        const unsigned low = __reduce_min_sync(0xffffffffu, tid < a.P ? load : 0xffffffffu);
        const unsigned high = __reduce_max_sync(0xffffffffu, load);
        if (lane == 0) {
          lows[warp] = low;
          highs[warp] = high;
        }
        __syncthreads();
        unsigned lo = lows[0], hi = highs[0];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) {
          lo = min(lo, lows[i]);
          hi = max(hi, highs[i]);
        }
        const int bin = hi > lo ? (int)((float)(load - lo) * (255.5f / (float)(hi - lo))) & 255 : 0;
        unsigned pos = 0;
        if (tid < a.P) pos = atomicAdd(&bins[bin], 1u);
        __syncthreads();
        const unsigned mine_bin = bins[tid];
        unsigned inc = mine_bin;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        if (lane == 31) scan[warp] = inc;
        __syncthreads();
        inc -= mine_bin;
#pragma unroll
        for (int i = 0; i < T / 32; ++i)
          if (i < warp) inc += scan[i];
        bins[tid] = inc;
        __syncthreads();
        if (tid < a.P) rank = (int)(bins[bin] + pos);
        __syncthreads();
        bins[tid] = 0;
      }
      if (tid < a.P) {
        a.ranks[(size_t)row_of_ranks * a.P + tid] = (uint8_t)rank;
        if (pass == 1 && round == 0) mine.z = rank;
        for (int k = 0; k < 1 << shift; ++k) {
          const long long i = (long long)(round + k) * a.P + rank;
          if (i >= n) break;
          int work;
          if (i < head_items) {
            work = part_work[i];
          } else {
            const unsigned x = (unsigned)i - (unsigned)head_items, at = per_group(x);
            const unsigned in = x - at * per_group.d;  // see grouped_tile
            const int e = from + (int)((int)at == groups - 1 ? per_last(in) : per_tile(in));
            work = pass == 0 ? (e < CACHED ? kv_work[e] : halves(kv[e])) * per_kv
                             : (e < CACHED ? q_work[e] : blocks(qs[e]));
          }
          load += pass == 0 ? work * a.half_cost + a.kv_cost : work * a.block_cost + a.q_cost;
          ++taken;
        }
      }
    }
    if (pass == 0)
      mine.x = taken;
    else
      mine.y = taken;
    shifts |= shift << (8 * pass);
  }
  if (tid < a.P) a.head->cta[tid] = mine;
  if (tid == 0) *reinterpret_cast<int4*>(a.head) = make_int4(n_parts, n_split, joins, shifts);
}

// -D = -rowsum(dO o O) and -L * log2(e) of one 128-row tile and head per block step;
// rows past the sequence's end get 0 and -inf, so that P is exactly 0 there. Bound by
// reading O and dO from HBM: D / 8 lanes per row, 16 bytes of each per lane, four rows
// in flight per lane before any arithmetic. The launch bound asks for the registers of
// that; without one the compiler kept fewer in flight (16384 rows, 32 heads, d = 128: 52 us,
// 59 without; 2048 rows in 16, 32/8 heads, the whole pass: 33.3 and 36.9).
// With DEAL, block 0 deals the gradient kernel's items meanwhile.
template <int D, bool DEAL>
__global__ void __launch_bounds__(256, DEAL ? 3 : 4) packed_preprocess_kernel(
    const __nv_bfloat16* O, const __nv_bfloat16* dO, const float* L, const uint8_t* plan,
    long long off_kv, float* ws_nD, float* ws_nL2, long long ws_rows, int total, int nseq, int Hq,
    int d, int trigger, const DealArgs deal) {
  constexpr int LPR = D / 8;        // lanes per row
  constexpr int RPB = 256 / LPR;    // rows per block step
  constexpr int U = 4;              // steps in flight
  static_assert(128 % (RPB * U) == 0, "whole rounds of steps per tile");
  __shared__ float sums[128];
  grid_wait();
  if (trigger) grid_launch_dependents();
  const PlanHead* head = reinterpret_cast<const PlanHead*>(plan);
  const bool ok = plan_matches(head, total, nseq, &g_packed_bwd_status);
  if (DEAL && blockIdx.x == 0) {
    deal_items(deal, ok ? head->tiles128 : 0);
    return;
  }
  if (!ok) return;
  const long long pairs = (long long)head->tiles128 * Hq;
  const int sub = threadIdx.x % LPR, r0 = threadIdx.x / LPR;
  for (long long i = blockIdx.x - DEAL; i < pairs; i += gridDim.x - DEAL) {
    const int e = (int)(i / Hq), h = (int)(i - (long long)e * Hq);
    const PlanTile s = reinterpret_cast<const PlanTile*>(plan + off_kv)[e];
    const int valid = s.y - s.z * 128;  // rows of this tile
    const size_t row0 = (size_t)s.x + (size_t)s.z * 128;
#pragma unroll
    for (int base = 0; base < 128; base += RPB * U) {
      uint4 a[U], b[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = base + u * RPB + r0;
        a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < valid && 8 * sub < d) {
          const size_t at = ((row0 + r) * Hq + h) * d;
          a[u] = reinterpret_cast<const uint4*>(O + at)[sub];
          b[u] = reinterpret_cast<const uint4*>(dO + at)[sub];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float acc = bf16_lo(a[u].x) * bf16_lo(b[u].x) + bf16_hi(a[u].x) * bf16_hi(b[u].x) +
                    bf16_lo(a[u].y) * bf16_lo(b[u].y) + bf16_hi(a[u].y) * bf16_hi(b[u].y) +
                    bf16_lo(a[u].z) * bf16_lo(b[u].z) + bf16_hi(a[u].z) * bf16_hi(b[u].z) +
                    bf16_lo(a[u].w) * bf16_lo(b[u].w) + bf16_hi(a[u].w) * bf16_hi(b[u].w);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
        if (sub == 0) sums[base + u * RPB + r0] = acc;
      }
    }
    float lse = 0.f;  // of row threadIdx.x; read before the barrier
    if ((int)threadIdx.x < min(valid, 128)) lse = L[(size_t)h * total + row0 + threadIdx.x];
    __syncthreads();
    if (threadIdx.x < 128) {
      const int r = threadIdx.x;
      const size_t w = (size_t)h * ws_rows + s.w + s.z * 128 + r;
      ws_nD[w] = -sums[r];
      ws_nL2[w] = r < valid ? -lse * kLog2e : -INFINITY;
    }
    __syncthreads();
  }
}

// dV and dK of the split key blocks: the sums of their parts, in order. One thread per row
// and eight columns; bound by the parts' way through L2 and, for few of them, by latency.
template <int D>
__global__ void __launch_bounds__(256) packed_join_kernel(
    const BwdDealHead* head, const BwdJoin* joins, const float* parts, __nv_bfloat16* dK,
    __nv_bfloat16* dV, long long lddk, long long lddv, float scale, int d) {
  constexpr int UNIT = 2 * 4 * (D / 8) * 32;  // threads of a key block
  constexpr size_t STRIDE = 2 * 128 * D;      // floats of a part
  grid_wait();
  grid_launch_dependents();
  const int n = head->joins * UNIT;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    const int lane = i & 31, c8 = (i >> 5) % (D / 8), warp = (i / (32 * (D / 8))) & 3;
    const int w = (i / (UNIT / 2)) & 1;
    const BwdJoin j = joins[i / UNIT];
    const int key = j.s.z * 128 + warp * 32 + lane;
    if (key >= j.s.y || 8 * c8 >= d) continue;
    const float4* x = reinterpret_cast<const float4*>(
                          parts + (size_t)j.slot * STRIDE + (size_t)(w * 4 + warp) * 32 * D) +
                      c8 * 64 + lane;
    float s[8] = {};
#pragma unroll 4
    for (int k = 0; k < j.parts; ++k) {
      const float4 a = x[k * (STRIDE / 4)], b = x[k * (STRIDE / 4) + 32];
      s[0] += a.x;
      s[1] += a.y;
      s[2] += a.z;
      s[3] += a.w;
      s[4] += b.x;
      s[5] += b.y;
      s[6] += b.z;
      s[7] += b.w;
    }
    const float mul = w == 0 ? 1.f : scale;
    __nv_bfloat16* out = (w == 0 ? dV : dK) + (j.s.x + key) * (w == 0 ? lddv : lddk) +
                         (size_t)j.head * d + 8 * c8;
    *reinterpret_cast<uint4*>(out) =
        make_uint4(pack_bf16(s[0] * mul, s[1] * mul), pack_bf16(s[2] * mul, s[3] * mul),
                   pack_bf16(s[4] * mul, s[5] * mul), pack_bf16(s[6] * mul, s[7] * mul));
  }
}

// Whether key blocks may be split: where there are fewer of them than SMs (the sequences'
// last tiles aside), and one may have many halves. The lengths are on the device only; so
// that is where one of a sequence of four times the mean length has more than kSplitFrom,
// or one of a sequence that is nearly the whole batch eight times as many. Where none is
// split after all, the look costs some 5 us (eight sequences of 500, 16/4 heads, d = 128: 65
// us, 60 without).
bool may_split(int total, int nseq, int Hq, int Hkv, int sms) {
  const long long most = ceil_div(total, 64), per_kv = Hq / Hkv;
  const long long likely = (4LL * ceil_div(total, nseq) + 63) / 64;
  return (long long)ceil_div(total, 128) * Hkv < sms &&
         ((likely < most ? likely : most) * per_kv > kSplitFrom ||
          most * per_kv > 8 * kSplitFrom);
}

int sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

template <int D>
cudaError_t launch_packed_bwd_d(const PackedBwdArgs& a, cudaStream_t stream) {
  const PlanLayout lay = plan_layout(a.nseq, a.total);
  const PackedBwdLayout ws = packed_bwd_layout(a.nseq, a.total, a.Hq);
  const long long ws_rows = ws.rows;
  uint8_t* const base = static_cast<uint8_t*>(a.workspace);
  float* const ws_nD = reinterpret_cast<float*>(base + ws.nD);
  float* const ws_nL2 = reinterpret_cast<float*>(base + ws.nL2);
  float* const parts = reinterpret_cast<float*>(base + ws.parts);
  const int sms = min(sm_count(), kMaxBwdCtas), per_kv = a.Hq / a.Hkv;
  const long long pairs = lay.cap[kKeyList] * a.Hq;
  const bool split = may_split(a.total, a.nseq, a.Hq, a.Hkv, sms);
  const long long items = pairs + lay.cap[kKeyList] * a.Hkv + (split ? ws.slots : 0);
  const unsigned ctas = (unsigned)(items < sms ? items : sms);
  DealArgs deal;
  deal.plan = static_cast<const uint8_t*>(a.plan);
  deal.off_kv = (long long)lay.off[kKeyList];
  deal.off_q = (long long)lay.off[1];
  deal.head = reinterpret_cast<BwdDealHead*>(base + ws.head);
  deal.joins = reinterpret_cast<BwdJoin*>(base + ws.joins);
  deal.items = reinterpret_cast<BwdItem*>(base + ws.items);
  deal.ranks = base + ws.ranks;
  deal.P = (int)ctas;
  deal.Hq = a.Hq;
  deal.Hkv = a.Hkv;
  deal.causal = a.causal;
  const int tiles = ceil_div(a.total, 128);
  deal.kgroup = heads_per_group(a.Hkv, tiles);
  deal.qgroup = round_up(heads_per_group(a.Hq, tiles), per_kv);
  deal.slots = ws.slots;
  // Fitted to the times of single items: a key block 3510 + 1596 per half at d = 128, 2561 +
  // 1431 at 64; a query block 2270 + 2028 per key block, 2000 + 2450.
  deal.half_cost = D == 128 ? 8 : 7;
  deal.kv_cost = D == 128 ? 18 : 13;
  deal.block_cost = D == 128 ? 10 : 12;
  deal.q_cost = D == 128 ? 11 : 10;
  cudaError_t e = launch_early(
      split ? packed_preprocess_kernel<D, true> : packed_preprocess_kernel<D, false>,
      (unsigned)((pairs < 8LL * sms ? pairs : 8LL * sms) + split), 256, 0, stream,
      static_cast<const __nv_bfloat16*>(a.O), static_cast<const __nv_bfloat16*>(a.dO), a.L,
      static_cast<const uint8_t*>(a.plan), (long long)lay.off[kKeyList], ws_nD, ws_nL2, ws_rows,
      a.total, a.nseq, a.Hq, a.d, pairs < sms ? 1 : 0, deal);
  if (e != cudaSuccess) return e;

  CUtensorMap mq, mk, mv, mdo, ml2, md, mdq, mdk, mdv;
  const long long ldo = (long long)a.Hq * a.d;
  const cuuint64_t dims[2] = {(cuuint64_t)ws_rows, (cuuint64_t)a.Hq};
  const cuuint64_t strides[1] = {(cuuint64_t)ws_rows * 4};
  const cuuint32_t box[2] = {64, 1};
  if (make_bf16_packed_map(&mq, a.Q, a.total, a.Hq, a.d, a.ldq, 64) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mk, a.K, a.total, a.Hkv, a.d, a.ldk, 128) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mv, a.V, a.total, a.Hkv, a.d, a.ldv, 128) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mdo, a.dO, a.total, a.Hq, a.d, ldo, 64) != CUDA_SUCCESS ||
      encode_tensor_map(&ml2, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, ws_nL2, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
      encode_tensor_map(&md, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, ws_nD, dims, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mdq, a.dQ, a.total, a.Hq, a.d, a.lddq) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mdk, a.dK, a.total, a.Hkv, a.d, a.lddk) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mdv, a.dV, a.total, a.Hkv, a.d, a.lddv) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  BwdParams p;
  p.d = a.d;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kLog2e;
  PackedBwdParams g;
  g.plan = static_cast<const uint8_t*>(a.plan);
  g.dQ = static_cast<__nv_bfloat16*>(a.dQ);
  g.dK = static_cast<__nv_bfloat16*>(a.dK);
  g.dV = static_cast<__nv_bfloat16*>(a.dV);
  g.lddq = a.lddq;
  g.lddk = a.lddk;
  g.lddv = a.lddv;
  g.nD = ws_nD;
  g.nL2 = ws_nL2;
  g.deal = deal.head;
  g.items = deal.items;
  g.ranks = deal.ranks;
  g.off_kv = deal.off_kv;
  g.off_q = deal.off_q;
  g.kgroup = deal.kgroup;
  g.qgroup = deal.qgroup;
  g.parts = parts;
  g.ws_rows = ws_rows;
  g.total = a.total;
  g.nseq = a.nseq;
  g.Hq = a.Hq;
  g.Hkv = a.Hkv;
  g.per_kv = per_kv;
  g.causal = a.causal;
  g.fill = a.fill;
  constexpr int smem = BwdSmem<D>::BYTES;
  auto kernel = split ? bwd_kernel<D, PackedBwd<true>> : bwd_kernel<D, PackedBwd<false>>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  g.trigger = (int)ctas < sms;  // see launch_as
  e = launch_early(kernel, ctas, KvCfg<D>::THREADS, smem, stream, mq, mk, mv, mdo,
                   ml2, md, mdq, mdk, mdv, p, g);
  if (e != cudaSuccess || !split) return e;
  return launch_early(packed_join_kernel<D>, (unsigned)(2 * sms), 256, 0, stream, deal.head,
                      deal.joins, parts, g.dK, g.dV, a.lddk, a.lddv, a.scale, a.d);
}

}  // namespace

cudaError_t launch_packed_backward(const PackedBwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_packed_bwd_d<128>(a, s) : launch_packed_bwd_d<64>(a, s);
}

cudaError_t packed_bwd_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_packed_bwd_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_packed_bwd_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
