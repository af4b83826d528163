// The forward kernel of exact attention: O = softmax(Q K^T * scale) V and the
// natural-log logsumexp L, two 128-row query tiles per CTA. It is shared by the
// dense forward pass, the forward pass over packed sequences and the prefix pass
// of decode attention, which differ in a geometry G: what a work item is, where
// its Q, K and V rows come from and where its results go.
//
// Method: "05_flash_attention.py", flash_attention_forward. For each query
// tile the key/value blocks are visited left to right; per row the kernel
// keeps a reference maximum m and the exponential sum l taken relative to it,
// forms P = exp(S - m), and adds P V to the output accumulator; whenever m
// moves, O and l are rescaled by exp(m_old - m_new). At the end O = O / l and
// L = m + log l. Under causal masking key blocks wholly to the right of a
// tile's last query are never visited, and the diagonal block masks k > q.
// The reference maximum is moved only when a row maximum exceeds it by more
// than 8 (base 2): until then P stays below 2^8 and O, l keep their common
// reference, so the result is the same up to rounding while most blocks need
// no rescaling of O. P is rounded to bf16 (2^-8 of a weight at most), the operand
// type of the full-rate products; l is summed in fp32 before that rounding.
//
// GB300 mapping (one persistent CTA per SM, 384 threads). The work items are
// (pair of 128-row query tiles, head); CTA c takes items c, 2P - 1 - c, 2P + c, ...
// of the launch-order list (P CTAs, heaviest items first within a group of heads).
//   warp 0       TMA producer: per item both Q tiles (one ring slot), then K_j
//                and V_j (128 keys each) into a ring shared by the two tiles; the
//                ring runs on across items, so the next item's Q and first blocks
//                arrive while the current item finishes
//   warp 1       MMA issuer (whole warp, one elected lane issues). Keys are
//                taken in steps of 64 (half a loaded block): S_t = Q_t K^T (TS:
//                Q_t read from TMEM) and O_t += P_t V (TS: P_t read from TMEM),
//                the two tiles alternating; S_t of step k+1 is issued right
//                after O_t += P_t V of step k, over the same columns
//   warps 4..7   softmax of tile 0, warps 8..11 softmax of tile 1: thread r
//                first moves row r of Q_t into TMEM, then owns query row r of its
//                tile (= TMEM lane r): reads the 64 S columns of a step with
//                tcgen05.ld, masks, updates (m, l) in base 2 (exp2 via
//                ex2.approx), writes P as bf16 over the first 32 of them,
//                rescales its O row when m moved, moves row r of the next
//                item's Q_t into TMEM and then runs the epilogue (O_t leaves
//                TMEM while the next item's first S_t is formed). While one
//                tile's softmax runs, the tensor cores work on the other.
// TMEM (512 columns at d = 128): Q0, Q1 (d/2 each, bf16 pairs), S0, S1 (64
// each), O0, O1 (d each). Scores, probabilities and the accumulators never
// leave the SM.
//
// A geometry G provides Params (a kernel argument), View (what the functions below
// get: the Params, or a copy with what the device had to look up), Item (one work
// item, a plain struct) and the functions
//   view(params)              read once at the kernel's start
//   items(g), item(g, i)      the work items (tile pair, head, ...) in launch order,
//                             dealt out in snake order; read one item ahead
//   segments, segment         instead of them (kSplit): what each CTA works on, an
//                             equal share of a long axis
//   steps(g, it, t)           64-key steps of tile t (tile 0 always has some)
//   keys(g, it)               keys of the item; steps past them are masked
//   causal(g), query(g, it, t, row)  the query position of a tile's row
//   place                     what load_kv needs to know of a block from memory: read
//                             one block ahead, so that the producer does not wait
//   load_q, load_kv           TMA loads of a Q tile / a 128-key block
//   tile_bytes, block_bytes   the bytes that they bring
//   store                     the epilogue of one warp's 32 rows
//   idle_warps                work of the warps that have no role
//   kEarly, trigger           launched with launch_early (see fa_launch.h), and whether
//                             the next kernel may start as early
//   kAlternate                both tiles of an item hold the same rows (see half_of),
//                             and store_joined writes the join of the two
//   status()                  the translation unit's device status word
//   kForeignTail              rows past the item's keys hold foreign values
#pragma once

#include "fa_internal.h"
#include "sm103.cuh"

namespace fa {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRescaleThreshold = 8.0f;  // base-2 units: P stays below 2^8

template <int D>
struct FwdCfg {
  static constexpr int BM = 128;                 // query rows per tile = TMEM lanes
  // Query tiles per CTA. TMEM would hold a third at d = 64, but with the deal's
  // wave quantization at the d = 64 workload sizes three tiles ran slower.
  static constexpr int TILES = 2;
  static constexpr int QUSES = (TILES + 1) / 2;  // ring uses holding an item's Q tiles
  static constexpr int SOFT0 = (TILES == 3) ? 2 : 4;  // first softmax warp
  static constexpr int BN = 128;                 // keys per loaded block (two halves of 64)
  static constexpr int KCH = D / 64;             // 128-byte column chunks per row
  static constexpr int CHUNK = 128 * 128;        // bytes of one chunk of a 128-row tile
  static constexpr int TILE = KCH * CHUNK;       // bytes of a Q, K or V tile
  static constexpr int HALF_ROWS = 64 * 128;     // bytes of 64 rows of one chunk
  // Ring of K/V blocks; its first use holds the two Q tiles until they are in TMEM.
  static constexpr int STAGES = (D == 128) ? 3 : 6;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = STAGES * TILE;
  static constexpr int OFF_EPI = 2 * STAGES * TILE;  // O staging, one area per softmax warp
  static constexpr int OFF_BAR = OFF_EPI + 4 * TILES * kStoreStageBytes;
  // barrier slots
  static constexpr int B_KVF = 0;                // + slot: the slot's copies landed
  static constexpr int B_KVE = STAGES;           // + slot: the slot may be refilled
  static constexpr int B_IN = 2 * STAGES;        // Q tiles in TMEM (256 arrivals)
  static constexpr int B_SF = B_IN + 1;          // + tile: S_t of the current step done
  static constexpr int B_PF = B_SF + TILES;      // + tile: P_t written (128 arrivals)
  // + tile + TILES * (item & 1): the tile's last O += P V done (for a tile with no steps:
  // the item's products done). Two slots: a softmax group signals the next item's Q before
  // it waits for this, and where its tile has no steps in the next item that item's
  // products finish without the group. One barrier could complete twice before the wait
  // and hide its phase; the item after the next needs the group first.
  static constexpr int B_PVD = B_PF + TILES;
  static constexpr int B_DRAIN = B_PVD + 2 * TILES;
  static constexpr int B_X = B_DRAIN + 1;        // kAlternate: both tiles' row sums written
  static constexpr int B_Y = B_DRAIN + 2;        // kAlternate: both tiles' O read out
  static constexpr int NBAR = B_DRAIN + 3;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;
  // TMEM columns: Q_t as bf16 pairs (the A operand of S_t = Q_t K^T), S_t of one
  // 64-key step (then P_t as bf16 pairs over its first 32 columns), O_t.
  static constexpr uint32_t COL_Q = 0;           // + (D / 2) * tile
  static constexpr uint32_t COL_S = 128;         // + 64 * tile
  static constexpr uint32_t COL_O = 128 + 64 * TILES;  // + D * tile
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr int THREADS = 32 * (SOFT0 + 4 * TILES);
  static_assert(COL_O + TILES * D <= TMEM_COLS, "TMEM budget");
  static_assert((D / 2) * TILES <= COL_S, "TMEM budget");
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct FwdParams {
  int d;             // head dimension (<= D; the tiles' columns past d are zero)
  float scale_log2;  // scale * log2(e)
};

// Bounded wait that ignores the abort flag: used only to let copies or MMAs
// already in flight land before the CTA exits.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitMaxCycles / 4) break;
  }
}

// 64-key steps a tile of rows [q0, q0 + 128) visits (0 if the tile is past n).
__device__ __forceinline__ int tile_steps(int q0, int n, int m, int causal) {
  if (q0 >= n) return 0;
  int nh = (m + 63) / 64;
  if (causal) nh = min(nh, (min(q0 + 127, n - 1)) / 64 + 1);  // keys k <= q
  return nh;
}

template <int D, class G>
__global__ void __launch_bounds__(FwdCfg<D>::THREADS, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
               const FwdParams p, const typename G::Params gp) {
  using Item = typename G::Item;
  using C = FwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + C::NBAR);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wc{abort_flag, G::status()};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&bar[C::B_KVF + s], 1);
      mbar_init(&bar[C::B_KVE + s], 1);
    }
    mbar_init(&bar[C::B_IN], 128 * C::TILES);
    for (int t = 0; t < C::TILES; ++t) {
      mbar_init(&bar[C::B_SF + t], 1);
      mbar_init(&bar[C::B_PF + t], 128);
      mbar_init(&bar[C::B_PVD + t], 1);
      mbar_init(&bar[C::B_PVD + C::TILES + t], 1);
    }
    mbar_init(&bar[C::B_DRAIN], 1);
    mbar_init(&bar[C::B_X], 128 * C::TILES);
    mbar_init(&bar[C::B_Y], 128 * C::TILES);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // A launch that may begin before the stream's previous kernel has ended: everything
  // above touches only this block's own state.
  if constexpr (G::kEarly) {
    grid_wait();
    if (G::trigger(gp)) grid_launch_dependents();
  }
  typename G::View g = G::view(gp);
  // Persistent: CTA c takes items snake_item(j, c, P), j = 0, 1, ... of the list of
  // (tile pair, head) items in launch order: heads a group at a time (their K/V
  // stay in L2 while the group runs), inside a group the heaviest tile pairs (the
  // last ones, under causal masking) first.
  const int P = gridDim.x, cta = blockIdx.x;
  int n_mine = 0;
  if constexpr (G::kSplit) {
    n_mine = G::segments(g, cta, P);
  } else {
    const int n_items = G::items(g);
    while (snake_item(n_mine, cta, P) < n_items) ++n_mine;
  }
  // Item j of this CTA.
  auto fetch = [&](int j) {
    if constexpr (G::kSplit)
      return G::segment(g, cta, P, j);
    else
      return G::item(g, snake_item(j, cta, P));
  };
  // With kAlternate the two tiles hold the same rows and take the halves of each
  // 128-key block in turn, so that one tile's rows keep both softmax groups busy.
  auto half_of = [](int t, int k) { return G::kAlternate ? 2 * k + t : k; };
  auto blocks = [](int nh) { return G::kAlternate ? nh : (nh + 1) / 2; };
  // The 64-key steps of each tile of an item (tile 0 always has some); returns the
  // steps of the longest tile.
  auto steps = [&](const Item& it, int (&nht)[C::TILES]) {
    int nh = 0;
#pragma unroll
    for (int t = 0; t < C::TILES; ++t) {
      nht[t] = G::steps(g, it, t);
      nh = max(nh, nht[t]);
    }
    return nh;
  };
  // Ring uses of item j: QUSES for its Q tiles (tiles 2u and 2u + 1 in the K and V
  // buffers of use u), then one per 128-key block of K, V. Every role counts them
  // (`ru`) and the steps of each tile identically.

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // Per item: the two Q tiles into the K and V buffers of one ring slot, then
    // K_j, V_j per block. The ring runs on across items, so the next item's Q and
    // first blocks load while the current item finishes.
    if (lane == 0 && n_mine > 0) {
      tma_prefetch_map(&tmQ);
      tma_prefetch_map(&tmK);
      tma_prefetch_map(&tmV);
      int ru = 0;
      bool ok = true;
      Item nxt = fetch(0);
      for (int j = 0; ok && j < n_mine; ++j) {
        const Item it = nxt;
        if (j + 1 < n_mine) nxt = fetch(j + 1);
        int nht[C::TILES];
        const int nkb = blocks(steps(it, nht));  // 128-key blocks
        auto place = G::place(g, it, 0);  // where the next block's keys are
        for (int u = 0; u < C::QUSES + nkb; ++u, ++ru) {
          const int s = ru % C::STAGES;
          if (ru >= C::STAGES &&
              !mbar_wait(&bar[C::B_KVE + s], ((ru / C::STAGES) & 1) ^ 1, wc)) {
            ok = false;
            break;
          }
          uint64_t* f = &bar[C::B_KVF + s];
          // Q tiles 2u, 2u + 1 (the second only if the CTA has it), or K and V
          const bool q_use = u < C::QUSES;
          const bool two = !q_use || 2 * u + 1 < C::TILES;
          if (q_use)
            mbar_arrive_expect_tx(f, (two ? 2 : 1) * G::template tile_bytes<C>(g));
          else
            mbar_arrive_expect_tx(f, G::template block_bytes<C>(g, it, u - C::QUSES));
          uint8_t* kdst = smem + C::OFF_K + s * C::TILE;
          uint8_t* vdst = smem + C::OFF_V + s * C::TILE;
          if (q_use) {
#pragma unroll
            for (int c = 0; c < C::KCH; ++c) {
              G::load_q(kdst + c * C::CHUNK, &tmQ, f, c * 64, g, it, 2 * u);
              if (two) G::load_q(vdst + c * C::CHUNK, &tmQ, f, c * 64, g, it, 2 * u + 1);
            }
          } else {
            const auto here = place;
            if (u + 1 < C::QUSES + nkb) place = G::place(g, it, u + 1 - C::QUSES);
            G::template load_kv<C>(kdst, vdst, &tmK, &tmV, f, g, it, u - C::QUSES, here);
          }
        }
      }
      // Let every copy this thread issued land before the CTA can exit.
      for (int r = max(0, ru - C::STAGES); r < ru; ++r)
        drain_wait(&bar[C::B_KVF + r % C::STAGES], (r / C::STAGES) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // Keys in steps of 64 (half a loaded block); the two tiles alternate:
    //   S_0(0) S_1(0) | O_0 += P_0(0) V, S_0(1), O_1 += P_1(0) V, S_1(1) | ...
    // S_t(k+1) overwrites P_t(k), read by the O_t product issued just before it
    // (tcgen05.mma instructions of one thread execute in order).
    if (n_mine > 0) {
      constexpr uint32_t kIdescS = idesc_bf16_f32(128, 64, false, false);
      constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, false, true);
      int ru = 0;                 // ring uses of earlier items
      int base[C::TILES] = {};    // each tile's steps in earlier items
      bool ok = true;
      Item nxt = fetch(0);
      for (int j = 0; ok && j < n_mine; ++j) {
        const Item it = nxt;
        int nht[C::TILES];
        const int nh = steps(it, nht), nkb = blocks(nh);
        // ring use of the block that holds half `u` of the item's keys
        auto use_of = [&](int u) { return ru + C::QUSES + (u >> 1); };
        auto scores = [&](int t, int k) {
          const int u = half_of(t, k);
          const uint64_t b_k = sdesc_sw128(
              smem_u32(smem + C::OFF_K + (use_of(u) % C::STAGES) * C::TILE + (u & 1) * C::HALF_ROWS),
              16, 1024);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * C::CHUNK + (kk & 3) * 32;
            umma_ts_w(tmem + C::COL_S + 64 * t, tmem + C::COL_Q + (D / 2) * t + kk * 8,
                      sdesc_add(b_k, off), kIdescS, kk > 0);
          }
          umma_commit_w(&bar[C::B_SF + t]);
        };
        auto pv = [&](int t, int k) {
          const int u = half_of(t, k);
          const uint64_t b_mn = sdesc_sw128(
              smem_u32(smem + C::OFF_V + (use_of(u) % C::STAGES) * C::TILE + (u & 1) * C::HALF_ROWS),
              C::CHUNK, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts_w(tmem + C::COL_O + D * t, tmem + C::COL_S + 64 * t + kk * 8,
                      sdesc_add(b_mn, kk * 2048), kIdescO, (k > 0 || kk > 0) ? 1u : 0u);
        };
        // Q_0, Q_1 in TMEM. (O_t of the previous item may still be being read out:
        // the O_t += P_t V product that overwrites it waits for P_t, which its
        // softmax warps write only after that.)
        if (!warp_wait(&bar[C::B_IN], j & 1, wc)) { ok = false; break; }
        if (lane == 0)  // the Q slots are free
          for (int u = 0; u < C::QUSES; ++u) mbar_arrive(&bar[C::B_KVE + (ru + u) % C::STAGES]);
        const int u1 = use_of(0);
        if (!warp_wait(&bar[C::B_KVF + u1 % C::STAGES], (u1 / C::STAGES) & 1, wc)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < C::TILES; ++t)
          if (nht[t] > 0) scores(t, 0);
        if (j + 1 < n_mine) nxt = fetch(j + 1);
        for (int k = 0; ok && k < nh; ++k) {
          // step k + 1 opens a block
          if (k + 1 < nh && (half_of(0, k + 1) & 1) == 0) {
            const int u = use_of(half_of(0, k + 1));
            if (!warp_wait(&bar[C::B_KVF + u % C::STAGES], (u / C::STAGES) & 1, wc)) { ok = false; break; }
          }
#pragma unroll
          for (int t = 0; t < C::TILES; ++t) {
            if (k >= nht[t]) continue;
            if (!warp_wait(&bar[C::B_PF + t], (base[t] + k) & 1, wc)) { ok = false; break; }
            tc_fence_after();
            pv(t, k);
            if (k + 1 < nht[t])
              scores(t, k + 1);
            else
              umma_commit_w(&bar[C::B_PVD + C::TILES * (j & 1) + t]);
          }
          // both tiles are done with a block once its second half's step is issued
          if (ok && (G::kAlternate || (k & 1) || k + 1 == nh))
            umma_commit_w(&bar[C::B_KVE + use_of(half_of(0, k)) % C::STAGES]);
        }
        // A tile with no steps (the second tile of a head's last pair when n mod 256
        // <= 128) is signalled once the item's products are done, so that its
        // softmax warps wait for the item's blocks to be consumed before they wait
        // for the next item's Q slot (whose earlier fill is one of those blocks).
#pragma unroll
        for (int t = 0; t < C::TILES; ++t)
          if (ok && nht[t] == 0) umma_commit_w(&bar[C::B_PVD + C::TILES * (j & 1) + t]);
        ru += C::QUSES + nkb;
#pragma unroll
        for (int t = 0; t < C::TILES; ++t) base[t] += nht[t];
      }
      umma_commit_w(&bar[C::B_DRAIN]);
      drain_wait(&bar[C::B_DRAIN], 0);
    }
  } else if (warp >= C::SOFT0) {
    // ------------------------------------------------------------ softmax
    const int t = (warp - C::SOFT0) >> 2;          // query tile of this warpgroup
    const int row = (warp & 3) * 32 + lane;        // row in the tile = TMEM lane
    const int row_thread = threadIdx.x & 127;      // thread of this warpgroup
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lane_base + C::COL_S + 64 * t;
    const uint32_t ocol = lane_base + C::COL_O + D * t;
    const float sl2 = p.scale_log2;
    int ru = 0, base_t = 0;  // ring uses and steps of tile t in earlier items
    // Row `row` of Q_t of the item whose Q tiles are ring use `rq` into TMEM: the
    // row's 16-byte pieces in the 128-byte-swizzled tile (piece j of a chunk row at
    // j ^ (row % 8)). The previous item's S_t products, the only readers of these
    // columns, are complete: this warp waited for each of them.
    auto move_q = [&](int rq) {
      const int uq = rq + (t >> 1);  // the ring use holding Q_t
      const int s = uq % C::STAGES;
      if (!warp_wait(&bar[C::B_KVF + s], (uq / C::STAGES) & 1, wc)) return false;
      const uint8_t* tile = smem + ((t & 1) == 0 ? C::OFF_K : C::OFF_V) + s * C::TILE;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t v[32];
        const uint8_t* src = tile + c * C::CHUNK + row * 128;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 x = *reinterpret_cast<const uint4*>(src + ((q ^ (row & 7)) << 4));
          v[4 * q] = x.x;
          v[4 * q + 1] = x.y;
          v[4 * q + 2] = x.z;
          v[4 * q + 3] = x.w;
        }
        tmem_st32(lane_base + C::COL_Q + (D / 2) * t + 32 * c, v);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bar[C::B_IN]);
      return true;
    };
    Item nxt{};
    if (n_mine > 0) nxt = fetch(0);
    bool ok = n_mine == 0 || move_q(0);
    for (int j = 0; ok && j < n_mine; ++j) {
      const Item it = nxt;
      int nht[C::TILES];
      const int nkb = blocks(steps(it, nht));
      const int nh_t = nht[t];
      const int m_keys = G::keys(g, it);
      const int qg = G::causal(g) ? G::query(g, it, t, row) : 0;
      float m_ref = -INFINITY;  // reference maximum of S * scale * log2(e)
      float l_run = 0.f;        // sum of exp2(S * scale * log2(e) - m_ref)
      for (int k = 0; ok && k < nh_t; ++k) {
        if (!warp_wait(&bar[C::B_SF + t], (base_t + k) & 1, wc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld32(scol, sr);
        tmem_ld32(scol + 32, sr + 32);
        tmem_ld_wait();
        reg_fence32(sr);
        reg_fence32(sr + 32);

        // Last visible column of this step for this row (ragged m, causal k <= q).
        const int ks = 64 * half_of(t, k);
        int lim = m_keys - 1 - ks;
        if (G::causal(g)) lim = min(lim, qg - ks);
        if (lim < 63) {
  #pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > lim) sr[c] = __float_as_uint(-INFINITY);
        }
        // Row maximum: eight chains of three-input maxima.
        float mx[8];
  #pragma unroll
        for (int e = 0; e < 8; ++e) mx[e] = __uint_as_float(sr[e]);
  #pragma unroll
        for (int c = 8; c < 64; c += 16)
  #pragma unroll
          for (int e = 0; e < 8; ++e)
            mx[e] = max3f(mx[e], __uint_as_float(sr[c + e]), __uint_as_float(sr[c + 8 + e]));
        const float rmax = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]),
                                 fmaxf(mx[6], mx[7])) * sl2;
        // Move the reference only when the row maximum passed it by the threshold.
        const bool move = rmax > m_ref + kRescaleThreshold;
        const float m_new = move ? rmax : m_ref;
        const float corr = move ? ex2(m_ref - m_new) : 1.f;  // 0 on the first step
        const float m_use = (m_new == -INFINITY) ? 0.f : m_new;  // no (-inf) - (-inf)
        m_ref = m_new;
        // P = exp2(S * scale * log2(e) - m) as bf16 pairs over this row's own S
        // columns.
        const uint64_t sl2x2 = f2pack(sl2, sl2);
        const uint64_t negm2 = f2pack(-m_use, -m_use);
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t pp[32];
  #pragma unroll
        for (int c = 0; c < 32; ++c) {
          const uint64_t x2 = ffma2(
              f2pack(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), sl2x2, negm2);
          float x0, x1;
          f2unpack(x2, x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          acc2[c & 3] = fadd2(acc2[c & 3], f2pack(p0, p1));
          pp[c] = pack_bf16(p0, p1);
        }
        // S_t(k) completing implies O_t += P_t(k-1) V completed (issued before it),
        // so the O row may be rescaled before this step's product is signalled.
        if (k >= 1 && __any_sync(0xffffffffu, move)) {
  #pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(ocol + 32 * c, o);
            tmem_ld_wait();
            reg_fence32(o);
  #pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
            tmem_st32(ocol + 32 * c, o);
          }
        }
        tmem_st32(scol, pp);
        tmem_st_wait();
        // V rows past the item's keys hold another sequence's values or whatever a
        // page held before, NaN perhaps, and 0 * NaN is NaN: the step that reads
        // them gets zeros. Both tiles' groups may write them (the same zeros).
        if constexpr (G::kForeignTail) {
          if (m_keys - ks < 64) {
            const int u = half_of(t, k);
            uint8_t* v = smem + C::OFF_V + ((ru + C::QUSES + (u >> 1)) % C::STAGES) * C::TILE +
                         (u & 1) * C::HALF_ROWS;
            for (int i = (m_keys - ks) * 8 + row_thread; i < 64 * 8; i += 128)
#pragma unroll
              for (int c = 0; c < C::KCH; ++c)
                *reinterpret_cast<uint4*>(v + c * C::CHUNK + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        mbar_arrive(&bar[C::B_PF + t]);
        float s0, s1, s2, s3, s4, s5, s6, s7;
        f2unpack(acc2[0], s0, s1);
        f2unpack(acc2[1], s2, s3);
        f2unpack(acc2[2], s4, s5);
        f2unpack(acc2[3], s6, s7);
        l_run = l_run * corr + (((s0 + s1) + (s2 + s3)) + ((s4 + s5) + (s6 + s7)));
      }

      // A tile with no steps waits for the end of the item's products first: only
      // then has the earlier fill of the next item's Q slot surely landed, so that
      // the slot's barrier is at most one phase behind the wait in move_q.
      uint64_t* const pvd = &bar[C::B_PVD + C::TILES * (j & 1)];
      if (ok && nh_t == 0 && !warp_wait(pvd + t, (j >> 1) & 1, wc)) { ok = false; break; }
      // The next item's Q_t goes in before this item's O_t comes out, so that the
      // next item's first S products run while the O rows are written.
      if (ok && j + 1 < n_mine && !move_q(ru + C::QUSES + nkb)) ok = false;
      // The item after is read behind that barrier's arrival, which is a release and would
      // wait for loads before it.
      if (j + 1 < n_mine) nxt = fetch(j + 1);
      // ---------------------------------------------------------- epilogue
      if constexpr (G::kAlternate) {
        // Both groups hold partial results of the same rows: they exchange the rows'
        // (m, l) through the second half of each warp's staging area (store_joined has
        // the first), and group t joins and writes columns [t D/2, (t + 1) D/2).
        if (!ok) break;
        if (!warp_wait(pvd, (j >> 1) & 1, wc) || !warp_wait(pvd + 1, (j >> 1) & 1, wc)) {
          ok = false;
          break;
        }
        uint8_t* mine = smem + C::OFF_EPI + (warp - C::SOFT0) * kStoreStageBytes;
        uint8_t* other = smem + C::OFF_EPI + ((warp - C::SOFT0) ^ 4) * kStoreStageBytes;
        *reinterpret_cast<float2*>(mine + 2048 + lane * 8) = make_float2(m_ref, l_run);
        mbar_arrive(&bar[C::B_X]);
        if (!warp_wait(&bar[C::B_X], j & 1, wc)) { ok = false; break; }
        tc_fence_after();
        const float2 o = *reinterpret_cast<const float2*>(other + 2048 + lane * 8);
        const float2 s0 = t == 0 ? make_float2(m_ref, l_run) : o;
        const float2 s1 = t == 0 ? o : make_float2(m_ref, l_run);
        G::template store_joined<D>(g, it, t, warp & 3, lane, lane_base + C::COL_O, s0, s1,
                                    nht[1] > 0, mine, &tmO, p.d);
        tc_fence_before();
        mbar_arrive(&bar[C::B_Y]);
        // the next item's products overwrite both accumulators
        if (!warp_wait(&bar[C::B_Y], j & 1, wc)) { ok = false; break; }
      } else if (ok && nh_t > 0) {
        if (!warp_wait(pvd + t, (j >> 1) & 1, wc)) { ok = false; break; }
        tc_fence_after();
        G::template store<D>(g, it, t, warp & 3, lane, ocol, m_ref, l_run,
                             smem + C::OFF_EPI + (warp - C::SOFT0) * kStoreStageBytes, &tmO, p.d);
        tc_fence_before();  // O_t read out before the next item's products overwrite it
      }
      ru += C::QUSES + nkb;
      base_t += nh_t;
    }
    if (lane == 0) bulk_wait_all();  // the stores have read the staging buffers
  } else {
    G::idle_warps(g, (warp - 2) * 32 + lane, 32 * (C::SOFT0 - 2), p.d);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace
}  // namespace fa
