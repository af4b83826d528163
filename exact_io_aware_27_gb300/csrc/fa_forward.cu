// The dense forward pass: the forward kernel (fa_forward.cuh) over Q, K, V
// [BH, n|m, d]. Work items are (pair of 128-row query tiles, head).
#include "fa_forward.cuh"

namespace fa {

__device__ unsigned int g_fwd_status;

namespace {

struct Dense {
  struct Params {
    float* L;
    int n, m, BH, causal, num_pairs, group;
  };
  using View = const Params&;
  FA_DEV static View view(const Params& g) { return g; }
  struct Item {
    int qs, bh;  // first query, head
  };
  FA_DEV static unsigned int* status() { return &g_fwd_status; }
  static constexpr bool kSplit = false, kAlternate = false, kEarly = false;
  static constexpr bool kForeignTail = false;  // TMA reads zeros past a head's rows
  FA_DEV static int items(const Params& g) { return g.num_pairs * g.BH; }
  // Heads a group at a time (their K/V stay in L2 while the group runs), inside a
  // group the heaviest tile pairs (the last ones, under causal masking) first.
  FA_DEV static Item item(const Params& g, int i) {
    int pair, bh;
    grouped_tile(i, g.BH, g.num_pairs, g.group, pair, bh);
    if (g.causal) pair = g.num_pairs - 1 - pair;
    return {pair * 256, bh};
  }
  FA_DEV static int steps(const Params& g, const Item& it, int t) {
    return tile_steps(it.qs + t * 128, g.n, g.m, g.causal);
  }
  FA_DEV static int keys(const Params& g, const Item&) { return g.m; }
  FA_DEV static int causal(const Params& g) { return g.causal; }
  FA_DEV static int query(const Params&, const Item& it, int t, int row) {
    return it.qs + t * 128 + row;
  }
  FA_DEV static void load_q(void* dst, const CUtensorMap* map, uint64_t* f, int col,
                            const Params&, const Item& it, int t) {
    tma_load_3d(dst, map, f, col, it.qs + t * 128, it.bh);
  }
  template <class C>
  FA_DEV static uint32_t tile_bytes(const Params&) {
    return C::TILE;
  }
  template <class C>
  FA_DEV static uint32_t block_bytes(const Params&, const Item&, int) {
    return 2 * C::TILE;
  }
  struct Place {};
  FA_DEV static Place place(const Params&, const Item&, int) { return {}; }
  template <class C>
  FA_DEV static void load_kv(uint8_t* kdst, uint8_t* vdst, const CUtensorMap* mk,
                             const CUtensorMap* mv, uint64_t* f, const Params&, const Item& it,
                             int block, Place) {
#pragma unroll
    for (int c = 0; c < C::KCH; ++c) {
      tma_load_3d(kdst + c * C::CHUNK, mk, f, c * 64, block * C::BN, it.bh);
      tma_load_3d(vdst + c * C::CHUNK, mv, f, c * 64, block * C::BN, it.bh);
    }
  }
  // O / l as bf16 through the warp's staging area and TMA (rows past n and the zero
  // columns past d are not written), and L.
  template <int D>
  FA_DEV static void store(const Params& g, const Item& it, int t, int warp, int lane,
                           uint32_t ocol, float m_ref, float l, uint8_t* stage,
                           const CUtensorMap* mo, int d) {
    const int row0 = it.qs + t * 128 + warp * 32, q = row0 + lane;
    tmem_rows_store<D>(ocol, 1.f / l, stage, mo, 0, row0, g.n, it.bh, d);
    if (q < g.n) g.L[(size_t)it.bh * g.n + q] = (m_ref + lg2(l)) * kLn2;
  }
  FA_DEV static void idle_warps(const Params&, int, int, int) {}
};

template <int D>
cudaError_t launch_fwd_d(const FwdArgs& a, cudaStream_t stream) {
  using C = FwdCfg<D>;
  CUtensorMap mq, mk, mv, mo;
  // Rows of d values; the 64-column boxes read zeros past d.
  if (make_bf16_head_map(&mq, a.Q, a.BH, a.n, a.d, C::BM) != CUDA_SUCCESS ||
      make_bf16_head_map(&mk, a.K, a.BH, a.m, a.d, C::BN) != CUDA_SUCCESS ||
      make_bf16_head_map(&mv, a.V, a.BH, a.m, a.d, C::BN) != CUDA_SUCCESS ||
      make_bf16_store_map(&mo, a.O, a.BH, a.n, a.d) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  FwdParams p;
  p.d = a.d;
  p.scale_log2 = a.scale * 1.44269504088896340736f;
  typename Dense::Params g;
  g.L = a.L;
  g.n = a.n;
  g.m = a.m;
  g.BH = a.BH;
  g.causal = a.causal;
  g.num_pairs = ceil_div(a.n, C::TILES * C::BM);
  g.group = heads_per_group(a.BH, g.num_pairs);
  cudaError_t e = cudaFuncSetAttribute(fwd_kernel<D, Dense>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // One CTA per SM (persistent), fewer when there are fewer items.
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const long long items = (long long)g.num_pairs * a.BH;
  const unsigned grid = (unsigned)(items < sms ? items : sms);
  fwd_kernel<D, Dense><<<grid, C::THREADS, C::SMEM, stream>>>(mq, mk, mv, mo, p, g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_forward(const FwdArgs& a, cudaStream_t s) {
  return a.d > 64 ? launch_fwd_d<128>(a, s) : launch_fwd_d<64>(a, s);
}

cudaError_t forward_read_status(unsigned int* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_fwd_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_fwd_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
