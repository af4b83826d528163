// The forward pass over packed sequences: the forward kernel (fa_forward.cuh) over
// Q [total, Hq, d] and K, V [total, Hkv, d], whose rows are sequences one after
// another; query head h reads key/value head h / (Hq / Hkv).
//
// The query heads of one key/value head share its keys, so up to eight of them
// (`heads`, the largest power of two that divides Hq / Hkv) share a tile: row r of a
// 128-row tile is head r % heads of query r / heads, and a tile pair covers
// 256 / heads queries. The work is the same for a long sequence, and less where tiles
// are cut off: by the end of a short sequence and by the causal diagonal (at 16
// sequences of 20 to 1151 rows, 32/8 heads, the products executed fall by 17 %).
// Work items are (tile pair of a sequence, head group), from the plan's list: head
// groups a few at a time, inside those the heaviest tiles of all sequences first, and
// the groups of one key/value head next to each other, so that its K and V are read
// once into L2.
//
// A sequence's last key block and last query tile run into the next sequence's rows
// (or into rows of no sequence): keys past the end are masked, their V rows are
// zeroed in shared memory before the product reads them (the forward kernel's
// kForeignTail), and query rows past the end stay in their own TMEM lanes and are
// not stored.
#include "fa_forward.cuh"
#include "fa_launch.h"
#include "fa_packed.cuh"

namespace fa {

__device__ unsigned int g_packed_status;

namespace {

// ONE_TILE: an item is one 128-row tile instead of a pair, and both softmax groups work on
// it, each on every other 64 keys (the forward kernel's kAlternate): for batches with few
// tile pairs, whose time is that of the longest item.
struct PackedParams {
  const uint8_t* plan;
  float* L;
  __nv_bfloat16* O;
  long long off_list;           // the list's place in the plan
  int total, nseq, Hq, per_kv, causal, group, fill;
  int list, head_shift;         // tiles of 256 >> list rows; heads = 1 << head_shift
  int trigger;
};

template <bool ONE_TILE>
struct Packed {
  using Params = PackedParams;
  struct View {
    const Params& p;
    int tiles, covered;
  };
  FA_DEV static View view(const Params& p) {
    const PlanHead* head = reinterpret_cast<const PlanHead*>(p.plan);
    const bool ok = plan_matches(head, p.total, p.nseq, status());
    return {p, ok ? (&head->tiles256)[p.list] : 0, ok ? head->covered : p.total};
  }
  struct Item {
    PlanTile s;  // sequence start, length, tile
    int h;       // first query head
  };
  FA_DEV static unsigned int* status() { return &g_packed_status; }
  FA_DEV static bool trigger(const Params& p) { return p.trigger; }
  static constexpr bool kSplit = false, kAlternate = ONE_TILE, kEarly = true;
  static constexpr bool kForeignTail = true;
  FA_DEV static int items(const View& g) { return g.tiles * (g.p.Hq >> g.p.head_shift); }
  FA_DEV static Item item(const View& g, int i) {
    int rank, h;
    grouped_tile(i, g.p.Hq >> g.p.head_shift, g.tiles, g.p.group, rank, h);
    return {reinterpret_cast<const PlanTile*>(g.p.plan + g.p.off_list)[rank],
            h << g.p.head_shift};
  }
  // First query of tile t, within the sequence.
  FA_DEV static int tile_query(const View& g, const Item& it, int t) {
    return (ONE_TILE ? it.s.z : 2 * it.s.z + t) * (128 >> g.p.head_shift);
  }
  FA_DEV static int query(const View& g, const Item& it, int t, int row) {
    return tile_query(g, it, t) + (row >> g.p.head_shift);
  }
  FA_DEV static int steps(const View& g, const Item& it, int t) {
    const int q0 = tile_query(g, it, t), n = it.s.y;
    if (q0 >= n) return 0;
    const int last = min(q0 + (128 >> g.p.head_shift), n) - 1;
    const int halves = (g.p.causal ? last : n - 1) / 64 + 1;
    return ONE_TILE ? (halves + 1 - t) / 2 : halves;
  }
  FA_DEV static int keys(const View&, const Item& it) { return it.s.y; }
  FA_DEV static int causal(const View& g) { return g.p.causal; }
  FA_DEV static void load_q(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                            const View& g, const Item& it, int t) {
    tma_load_3d(dst, map, f, col, it.h, it.s.x + tile_query(g, it, t));
  }
  template <class C>
  FA_DEV static uint32_t tile_bytes(const View&) {
    return C::TILE;
  }
  template <class C>
  FA_DEV static uint32_t block_bytes(const View&, const Item&, int) {
    return 2 * C::TILE;
  }
  struct Place {};
  FA_DEV static Place place(const View&, const Item&, int) { return {}; }
  template <class C>
  FA_DEV static void load_kv(uint8_t* kdst, uint8_t* vdst, const CUtensorMap* mk,
                             const CUtensorMap* mv, uint64_t* f, const View& g, const Item& it,
                             int block, Place) {
    const int hk = it.h / g.p.per_kv, row = it.s.x + block * C::BN;
#pragma unroll
    for (int c = 0; c < C::KCH; ++c) {
      tma_load_3d(kdst + c * C::CHUNK, mk, f, c * 64, hk, row);
      tma_load_3d(vdst + c * C::CHUNK, mv, f, c * 64, hk, row);
    }
  }
  template <int D>
  FA_DEV static void store(const View& g, const Item& it, int t, int warp, int lane, uint32_t ocol,
                           float m_ref, float l, uint8_t* stage, const CUtensorMap* mo, int d) {
    const int sh = g.p.head_shift, q0 = tile_query(g, it, t) + ((warp * 32) >> sh);
    const int row0 = it.s.x + q0, valid = (it.s.y - q0) << sh;
    packed_rows_store<D>(ocol, 1.f / l, stage, mo, it.h, row0, valid, 0, d, g.p.O,
                         (long long)g.p.Hq * d, sh);
    if (lane < valid)
      g.p.L[(size_t)(it.h + (lane & ((1 << sh) - 1))) * g.p.total + row0 + (lane >> sh)] =
          (m_ref + lg2(l)) * kLn2;
  }
  // The same from the two halves of the keys: (m, l) = s0 with O in columns ocol, s1 with
  // O in ocol + D (nothing there where `second` is false). The join is written back over
  // group t's half of the columns [t D/2, (t + 1) D/2), which that group stores.
  template <int D>
  FA_DEV static void store_joined(const View& g, const Item& it, int t, int warp, int lane,
                                  uint32_t ocol, float2 s0, float2 s1, bool second,
                                  uint8_t* stage, const CUtensorMap* mo, int d) {
    const int sh = g.p.head_shift, q0 = tile_query(g, it, t) + ((warp * 32) >> sh);
    const int row0 = it.s.x + q0, valid = (it.s.y - q0) << sh;
    const float m = second ? fmaxf(s0.x, s1.x) : s0.x;
    const float ref = m == -INFINITY ? 0.f : m;
    const float f0 = ex2(s0.x - ref), f1 = second ? ex2(s1.x - ref) : 0.f;
    const float l = second ? s0.y * f0 + s1.y * f1 : s0.y * f0;
    const uint32_t mine = ocol + t * (D / 2);
    if (valid > 0) {  // warp-uniform
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        uint32_t x[32], y[32];
        tmem_ld32(mine + c, x);
        if (second) tmem_ld32(mine + D + c, y);
        tmem_ld_wait();
        reg_fence32(x);
        if (second) reg_fence32(y);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          float v = __uint_as_float(x[e]) * f0;
          if (second) v += __uint_as_float(y[e]) * f1;
          x[e] = __float_as_uint(v);
        }
        tmem_st32(mine + c, x);
      }
      tmem_st_wait();
    }
    packed_rows_store<D / 2, 1>(mine, 1.f / l, stage, mo, it.h, row0, valid, t * (D / 2), d, g.p.O,
                             (long long)g.p.Hq * d, sh);
    if (t == 0 && lane < valid)
      g.p.L[(size_t)(it.h + (lane & ((1 << sh) - 1))) * g.p.total + row0 + (lane >> sh)] =
          (ref + lg2(l)) * kLn2;
  }
  // Rows that no sequence covers: O = 0 and L = -inf (what attention to no key
  // gives), where the caller asked for it.
  FA_DEV static void idle_warps(const View& g, int thread, int threads, int d) {
    const long long t = (long long)blockIdx.x * threads + thread;
    const long long nt = (long long)gridDim.x * threads;
    const Params& p = g.p;
    if (p.fill & 1) zero_rows(p.O, g.covered, p.total, p.Hq * d, (long long)p.Hq * d, t, nt);
    if (p.fill & 2) {
      const long long rest = p.total - g.covered;
      for (long long i = t; i < rest * p.Hq; i += nt)
        p.L[(i / rest) * p.total + g.covered + i % rest] = -INFINITY;
    }
  }
};

template <int D>
cudaError_t launch_packed_d(const PackedFwdArgs& a, cudaStream_t stream) {
  using C = FwdCfg<D>;
  CUtensorMap mq, mk, mv, mo;
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int sh = 0;  // heads that share a tile: 1 << sh
  while (sh < 3 && a.Hq / a.Hkv % (2 << sh) == 0) ++sh;
  // Fewer pairs than SMs (the sequences' last pairs aside): single tiles. There is no list
  // of 16-row tiles. One sequence of 2000 rows, 8/1 heads, d = 128: 19.6 us in single tiles,
  // 31.9 in pairs; 4000 rows, 4/1 heads: 33.1, 58.3; three of 1000, 8/2, d = 64: 11.6, 16.4.
  // Short sequences have few keys to share out, and the join costs: one of 472 rows, 32/8,
  // 11.1 and 11.7; eight of 100, 16/8, 8.6 and 7.8. So from a mean length of 512. With one
  // to two pairs an SM their number comes out uneven, and single tiles win from about 1024:
  // five of 9000 rows in all, 8/8, 60.9 and 70.3; six of 3312, 24/8, 35.1 and 32.4; one of
  // 4096, 32/8 (3.4 pairs), 124 and 112.
  const long long pairs = (long long)ceil_div(a.total, 256 >> sh) * (a.Hq >> sh);
  const bool one = pairs < sms ? a.total / 512 >= a.nseq
                               : pairs < 2LL * sms && a.total / 1024 >= a.nseq;
  if (one && sh == 3) sh = 2;
  if (make_bf16_packed_map(&mq, a.Q, a.total, a.Hq, a.d, a.ldq, C::BM >> sh, 1 << sh) !=
          CUDA_SUCCESS ||
      make_bf16_packed_map(&mk, a.K, a.total, a.Hkv, a.d, a.ldk, C::BN) != CUDA_SUCCESS ||
      make_bf16_packed_map(&mv, a.V, a.total, a.Hkv, a.d, a.ldv, C::BN) != CUDA_SUCCESS ||
      make_bf16_packed_store_map(&mo, a.O, a.total, a.Hq, a.d, (long long)a.Hq * a.d, 1 << sh) !=
          CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  FwdParams p;
  p.d = a.d;
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  PackedParams g;
  g.plan = static_cast<const uint8_t*>(a.plan);
  g.L = a.L;
  g.O = static_cast<__nv_bfloat16*>(a.O);
  g.total = a.total;
  g.nseq = a.nseq;
  g.Hq = a.Hq;
  g.per_kv = a.Hq / a.Hkv;
  g.causal = a.causal;
  g.fill = a.fill;
  const int list = sh + (one ? 1 : 0);
  g.list = list;
  g.head_shift = sh;
  const PlanLayout lay = plan_layout(a.nseq, a.total);
  g.off_list = (long long)lay.off[list];
  // Whole key/value heads per group: as many as fill eight waves (the plan's tile count is
  // known on the device only; the rows give it up to the sequences' last tiles), or all
  // whose K and V fit half of L2: the fewer groups, the better the deal comes out (16384
  // rows, 32/8 heads, d = 128 in two groups: the busiest CTA had 14 % more than the mean).
  const long long fit = (64LL << 20) / ((long long)a.total * a.d * 4);
  const int heads = a.Hq >> sh;
  g.group = round_up(heads_per_group(heads, ceil_div(a.total, 256 >> list)), g.per_kv >> sh);
  if (fit * (g.per_kv >> sh) > g.group)
    g.group = fit >= a.Hkv ? heads : (int)fit * (g.per_kv >> sh);
  auto kernel = one ? fwd_kernel<D, Packed<true>> : fwd_kernel<D, Packed<false>>;
  cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const long long items = lay.cap[list] * heads;
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  g.trigger = (int)grid < sms;  // see launch_as
  return launch_early(kernel, grid, C::THREADS, C::SMEM, stream, mq, mk, mv, mo, p, g);
}

}  // namespace

cudaError_t launch_packed_forward(const PackedFwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_packed_d<128>(a, s) : launch_packed_d<64>(a, s);
}

cudaError_t packed_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_packed_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_packed_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
